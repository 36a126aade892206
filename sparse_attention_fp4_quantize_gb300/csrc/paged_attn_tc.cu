// The tile kernel of csa2_paged_attn_fp8 and csa2_paged_attn_fp4: prompts, and whatever else
// brings more rows per KV head than the split kernels' row tiles hold.
//
// A unit is 256 rows of one (request, KV head), two sub-tiles of 128, against
// tiles of 128 keys: 2 x 2 x 128 x 128 x D MACs per key tile on tcgen05 in f16
// with fp32 accumulators in TMEM.  Per key tile and sub-tile
//   S = Q . K^T      (M = 128 rows, N = 128 keys; Q and K tiles in shared memory, Q of 64
//                    channels over the 4-bit cache in TMEM)
//   P = f16 of the softmax weights, written over S in TMEM
//   O += P . V       (M = 128 rows, N = D; A = P from TMEM, V tile in shared memory)
// The codes become f16 once per CTA and key tile; both sub-tiles use them.
// K is read K-major and V MN-major from the same core-matrix layout, so one
// conversion serves both.  Roles (16 warps, registers shared out by warpgroup):
//   warps 0-3, 4-7   softmax of sub-tile 0, 1: thread = row (TMEM lane), so the
//                    row's maximum and sum need no exchange; also load Q and
//                    store the output
//   warps 8-11       bring codes (a key tile ahead; E4M3 into a staging buffer of their own,
//                    as the registers for them are the softmax's), convert, store
//   warps 12, 13     issue the MMAs of sub-tile 0, 1, taking turns
//   warp 14          works out the CTA's segments, a few ahead of the others
// While one sub-tile's softmax runs, the tensor cores have the other's products.
// The running references M, Mv (paged_attn.cu; the 4-bit cache has no Mv) move only when a
// tile's scores exceed them far enough to matter to f16, so most tiles need no maximum and O
// in TMEM is rescaled rarely.
//
// Bound by the chain softmax -> hand-over -> products -> hand-over of a sub-tile, which the
// other sub-tile's fills only in part.  The products of a key tile take 2048 cycles (64 per
// M 128 N 128 K 16); of the 3500 that it takes (clock64 in a copy), a sub-tile's softmax
// 1340 (128 exponentials, at 4 cycles per warp, are 512), waking the issuing warp 110, the
// lock 340 (an atomic behind the converters' stores), its 16 products 1050 to issue and
// 450 more until S is seen.  Of 64 channels, with half the products: 1280, 110, 390, 520, 440.
// 3 prompts of up to 4096 tokens on up to 8192, 32 heads of 128 over 8: 773 us over 8 bits,
// 735 over 4, 64 channels over 4 bits 637.
// The issuing warps run with all lanes and elect one for the products, so that descriptors
// stay in uniform registers: as one thread's work each product waited for them to be moved
// there, 94 cycles a product instead of 42 of 64 channels (845 against 783 us over 8 bits, 818
// against 761 over 4; 730 against 654 of 64 channels).  Tried and slower: P handed over in
// two halves of 64 keys (784 against 734 us), E4M3 codes kept in
// registers instead of staged (934 against 906 then; over 4 bits the same), the lock given up
// with half of S to go (750 against 741), before S (772 against 760) or left out (792
// against 745), strict turns by mbarriers in its place (771 against 745), waits that poll
// before they sleep (828 against 753 with 16 polls), S and P in halves of 64 keys that take
// turns in TMEM (789 against 735: a product of N 64 reads all of Q and takes 59 cycles, not 32), a
// row's keys shared by two warps that serve the sub-tiles in turn (820 against 734: two
// warps together need 1080 cycles for what one does in 1340, and 600 to come to the next).
#include "fp4.cuh"
#include "paged_attn.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kSoftWarps = 8, kConvWarps = 4, kMmaWarp = kSoftWarps + kConvWarps;
constexpr int kTcThreads = 512;              // four warpgroups, as the register shares go by warpgroup
// Registers per thread: 512 x 128 at launch; the softmax warpgroups, which hold
// a row's 128 scores, take what the others give up (over the 8-bit cache the converters give up
// less: with 72 its softmax spills).
constexpr int kLaunchRegs = 128;
template <bool FP4>
struct Regs {
    static constexpr int SOFT = FP4 ? 184 : 176, CONV = FP4 ? 72 : 80, MMA = CONV;
    static_assert(kLaunchRegs * kTcThreads == 65536, "the launch's registers are an SM's");
    static_assert(2 * SOFT + CONV + MMA <= 4 * kLaunchRegs, "register shares exceed the launch's");
    static_assert(SOFT >= kLaunchRegs && CONV <= kLaunchRegs && MMA <= kLaunchRegs,
                  "setmaxnreg.inc may not ask for fewer than the launch's, .dec not for more (an illegal instruction)");
    static_assert(SOFT % 8 == 0 && CONV % 8 == 0 && MMA % 8 == 0 && CONV >= 24 && MMA >= 24 && SOFT <= 256,
                  "setmaxnreg takes multiples of 8 from 24 to 256");
};
// A wait gives up after that many naps, which an arrival ends; the hardware cuts them to 6 us
// whatever is asked for (measured).  Within a key tile, of 2 us, 26 ms; for a segment, which may be 2^23 tiles
// (2^30 keys) long, 50 s: where something is lost the waits within a tile end all others.
constexpr uint32_t kPolls = 4096, kSegPolls = 1u << 23, kNap = 500000;
constexpr uint32_t kLockPolls = 1u << 24;
constexpr float kSlack = 14 - kUp;           // log2: how far a tile may exceed a reference before it moves (P < 2^(kUp + kSlack + 1))
constexpr float kSpread = 64.0f;             // log2: how far scales may lie apart in the common case
constexpr float kMostP = 65000.0f, kMostL = 1e30f;   // its bounds on a tile's sum of P (f16 ends at 65504) and gain of l
constexpr float kMostRaise = 0x1p64f;        // and on the sum where a higher Mv is tried
constexpr int kMetas = 4;                    // key tiles whose scales are kept

struct TileMeta {
    float ks[8], vs[8], lg[8], rv[8];        // scales of the 16-key groups; log2 of 2^kUp v's, its reciprocal
    uint32_t missing[4];                     // per converting warp: its groups that are not stored (a bit each)
};

// A piece of a unit.  One warp works out the CTA's segments and hands them to the
// others through a ring in shared memory.
constexpr int kSegs = 4;
struct alignas(16) Segment {
    Request rq;
    Place pl;
    int b, tb;                               // request, end of its key tiles [pl.tile, tb) of pl.tiles
    int rows, low;                           // rows of the request and KV head (0: no more segments); lowest key that the unit sees
    __device__ __forceinline__ int key0() const { return low & ~(kTcKeys - 1); }               // of its first tile
};

template <int D>
struct Lay {
    static constexpr uint32_t GROUP = D * 16;            // core matrices of 8 rows: D / 8 x 128 bytes
    static constexpr uint32_t Q = 128 * D * 2, KV = kTcKeys * D * 2;
    static constexpr uint32_t OFF_Q = 0, OFF_K = 2 * Q, OFF_V = OFF_K + 2 * KV, OFF_STAGE = OFF_V + 2 * KV, OFF_META = OFF_STAGE + KV,
                              OFF_SEG = OFF_META + kMetas * sizeof(TileMeta), OFF_BAR = OFF_SEG + kSegs * sizeof(Segment);
    static constexpr int BARS = 29;
    static constexpr uint32_t USED = OFF_BAR + BARS * 8 + 12;
    static constexpr uint32_t SMEM = USED + 128 > 120 * 1024 ? USED + 128 : 120 * 1024;   // one CTA per SM (TMEM)
    static constexpr uint32_t COL_S = 0, COL_O = 256, COL_Q = COL_O + 2 * D;   // TMEM columns: S0, S1 (P over them), O0, O1, and Q0, Q1 where there is room
    static constexpr bool TMEM_Q = COL_Q + D <= 512;
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

template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded wait of one thread that also gives up once another has raised the
// abort word; and of a whole warp, every lane of which gets the same answer.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int *abort_word, uint32_t polls = kPolls) {
    uint32_t ok;                             // most waits are over before they begin: asked without going to sleep
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    for (uint32_t i = 0; i < polls; ++i) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(kNap)
            : "memory");
        if (ok) return true;
        if (*abort_word) break;
    }
    *abort_word = 1;
    return false;
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_word, uint32_t polls = kPolls) {
    return __all_sync(0xFFFFFFFFu, wait_one(bar, parity, abort_word, polls));
}

// Logit factor of a key: not 0, so that a hidden score of -inf stays -inf.
__device__ __forceinline__ float factor(float zf, float ks) { return fmaxf(zf * ks, 1e-38f); }

// The CTA's segments in order.
struct Walk {
    int64_t at, stop, base, unit;            // place of the line, its end; first places of the request, of the unit
    Request rq;
    TcWork::Rows rows;
    int b, h;                     // h < 0: before the first segment
    __device__ __forceinline__ Walk(const PagedAttnArgs &a, const Plan &p, int cta)
        : at(cta * p.share), stop(min(p.total, at + p.share)), base(p.base), rows(a.G), b(p.b), h(-1) {}
    __device__ __forceinline__ bool next(const PagedAttnArgs &a, Segment &s) {
        if (at >= stop) return false;
        if (h < 0) {
            rq = request_of(a, b);
            s.pl = TcWork::place(a, rq, at - base, rows);
            h = s.pl.h;
        } else {                                          // the row tile, head or request after the last one
            rows.next();
            if (rows.r0 >= rq.n * a.G) {
                rows = TcWork::Rows(a.G);
                if (++h == a.Hkv) {
                    h = 0;
                    do {
                        if (++b >= a.B) return false;
                        rq = request_of(a, b);
                    } while (!TcWork::mine(a, rq));
                }
            }
            s.pl.h = h;
            s.pl.r0 = rows.r0;
            s.pl.tile = 0;
            s.pl.tiles = TcWork::unit_places(a, rq, rows);
        }
        unit = at - s.pl.tile;
        at = min(stop, unit + s.pl.tiles);
        s.rq = rq;
        s.b = b;
        s.tb = (int)(at - unit) - kTcCost;
        s.pl.tile = max(0, s.pl.tile - kTcCost);             // from places to tiles
        s.pl.tiles -= kTcCost;
        s.rows = rq.n * a.G;
        s.low = TcWork::low_key(a, rq, rows);
        return true;
    }
};

template <int D, bool HALF, bool FP4>
__global__ void __launch_bounds__(kTcThreads, 1) paged_attn_tc_kernel(PagedAttnArgs a) {
    using L = Lay<D>;
    constexpr bool TMEM_Q = FP4 && L::TMEM_Q;            // S reads Q from tensor memory, which halves what it asks of shared memory
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((128u - (tc::smem_u32(smem_raw) & 127u)) & 127u);
    __shared__ int64_t s_sum[kTcThreads / 32];
    __shared__ Found s_found;
    const int tid = threadIdx.x, warp = __shfl_sync(ALL, tid >> 5, 0), lane = tid & 31;
    const uint32_t sb = tc::smem_u32(smem);
    TileMeta *metas = reinterpret_cast<TileMeta *>(smem + L::OFF_META);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_BAR + L::BARS * 8);
    volatile int *abort_word = reinterpret_cast<volatile int *>(smem + L::OFF_BAR + L::BARS * 8 + 4);
    unsigned int *tensor_lock = reinterpret_cast<unsigned int *>(smem + L::OFF_BAR + L::BARS * 8 + 8);
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
    auto segfull = [&](int i) { return bar0 + 8u * (21 + i); };
    auto segempty = [&](int i) { return bar0 + 8u * (25 + i); };
    Segment *segs = reinterpret_cast<Segment *>(smem + L::OFF_SEG);
    const float NEG_INF = __int_as_float(0xff800000);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(kfull(i), kConvWarps);
            tc::mbar_init(kempty(i), 2);
            tc::mbar_init(vfull(i), kConvWarps);
            tc::mbar_init(vempty(i), 2);
            tc::mbar_init(qfull(i), 4);
            tc::mbar_init(sfull(i), 1);
            tc::mbar_init(pfull(i), 4);
            tc::mbar_init(ofull(i), 1);
        }
        for (int i = 0; i < kMetas; ++i) tc::mbar_init(mfull(i), kConvWarps);
        tc::mbar_init(drain, 2);
        for (int i = 0; i < kSegs; ++i) {
            tc::mbar_init(segfull(i), 1);
            tc::mbar_init(segempty(i), kSoftWarps + kConvWarps + 2);   // each warp that reads it
        }
        *abort_word = 0;
        *tensor_lock = 0;
        tc::mbar_init_fence();
    }
    if (warp == 0) tc::tmem_alloc(tmem_slot, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = __shfl_sync(ALL, *tmem_slot, 0);
    pdl_wait();
    pdl_launch_dependents();
    const Plan plan = plan_of<TcWork>(a, blockIdx.x, gridDim.x, 1, s_sum, &s_found);
    bool run = true;
    uint32_t n_seg = 0;
    // The next segment, of a whole warp.  False: none, or given up.
    auto next_seg = [&](Segment &s) -> bool {
        const uint32_t i = n_seg % kSegs, par = (n_seg / kSegs) & 1;
        ++n_seg;
        if (!wait_bar(segfull(i), par, abort_word, kSegPolls)) return false;
        s = segs[i];
        __syncwarp();
        if (lane == 0) arrive(segempty(i));
        return __shfl_sync(ALL, s.rows, 0) > 0;
    };

    if (warp >= kMmaWarp) {
        // ---- the MMAs, one warp per sub-tile: the waits of one, each worth 1.5 products
        // of idle tensor cores, overlap the other's products.  S of the next key tile goes
        // out behind P V of this one, which it may only overwrite then: the products of one
        // thread run in order.  The two take turns by a lock, P V and S at a time:
        // interleaved, both sub-tiles would get their scores late and at once, and the
        // softmaxes would run side by side and then the tensor cores alone.  A sub-tile
        // without rows in the segment only hands the buffers on.
        fewer_regs<Regs<FP4>::MMA>();
        const int sub = warp - kMmaWarp;
        if (warp == kMmaWarp + 2 && lane == 0) {
            // ---- the segments, and one of no rows behind the last
            Walk walk(a, plan, blockIdx.x);
            JoinUnit *join = a.join_tc + blockIdx.x;
            join->last = -1;
            for (bool more = true; more; ++n_seg) {
                Segment s = {};
                do more = walk.next(a, s);
                while (more && s.tb <= 0);
                if (!more) s.rows = 0;
                if (more && s.pl.tile == 0 && s.tb < s.pl.tiles)
                    *join = {s.rq.row0, s.pl.h, s.pl.r0, s.rows, (int)((walk.unit + kTcCost + s.pl.tiles - 1) / plan.share), {0, 0}};
                const uint32_t i = n_seg % kSegs;
                if (!wait_one(segempty(i), ((n_seg / kSegs) & 1) ^ 1, abort_word, kSegPolls)) break;
                segs[i] = s;
                arrive(segfull(i));
            }
        }
        if (sub < 2) {
            constexpr uint32_t idesc_s = tc::idesc_f16_f32(128, kTcKeys, false, false);
            constexpr uint32_t idesc_o = tc::idesc_f16_f32(128, D, false, true);
            const uint64_t dq = tc::desc_noswizzle(sb + L::OFF_Q + sub * L::Q, 128, L::GROUP);
            const uint64_t dk = tc::desc_noswizzle(sb + L::OFF_K, 128, L::GROUP);
            const uint64_t dv = tc::desc_noswizzle(sb + L::OFF_V, L::GROUP, 128);
            const uint32_t ts = tmem + L::COL_S + sub * 128, to = tmem + L::COL_O + sub * D;
            const uint32_t lock_at = tc::smem_u32(tensor_lock);
            uint32_t nk = 0, nq = 0, np = 0;             // key tiles, segments with this sub-tile, its P tiles so far
            auto lock = [&]() -> bool {
                for (uint32_t i = 0; i < kLockPolls; ++i) {
                    uint32_t held = 1;
                    if (lane == 0)
                        asm volatile("atom.relaxed.cta.shared::cta.cas.b32 %0, [%1], 0, 1;" : "=r"(held) : "r"(lock_at));
                    if (__any_sync(ALL, held == 0)) return true;
                    if (__any_sync(ALL, *abort_word)) break;
                }
                *abort_word = 1;
                return false;
            };
            auto unlock = [&]() { asm volatile("st.relaxed.cta.shared::cta.b32 [%0], 0;" ::"r"(lock_at)); };
            auto issue_s = [&](uint32_t tile) {
                const uint32_t q = (uint32_t)dq, k = (uint32_t)dk + (tile & 1) * (L::KV / 16);
                if (tc::elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        if constexpr (TMEM_Q) tc::mma_f16_ta_lo(ts, tmem + L::COL_Q + sub * (D / 2) + ks * 8, k + ks * 16, (uint32_t)(dk >> 32), idesc_s, ks > 0);
                        else tc::mma_f16_lo(ts, q + ks * 16, k + ks * 16, (uint32_t)(dk >> 32), idesc_s, ks > 0);
                    }
                    tc::commit(sfull(sub));
                    tc::commit(kempty(tile & 1));
                    unlock();
                }
            };
            auto issue_o = [&](uint32_t tile, bool first) {
                const uint32_t v = (uint32_t)dv + (tile & 1) * (L::KV / 16);
                if (tc::elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kTcKeys / 16; ++ks)
                        tc::mma_f16_ta_lo(to, ts + ks * 8, v + ks * (L::GROUP / 8), (uint32_t)(dv >> 32), idesc_o, !first || ks > 0);
                    tc::commit(ofull(sub));
                    tc::commit(vempty(tile & 1));
                }
            };
            auto wait_k = [&](uint32_t tile) { return wait_bar(kfull(tile & 1), (tile >> 1) & 1, abort_word); };
            auto wait_v = [&](uint32_t tile) { return wait_bar(vfull(tile & 1), (tile >> 1) & 1, abort_word); };
            auto wait_q = [&]() { return wait_bar(qfull(sub), nq++ & 1, abort_word); };
            auto wait_p = [&]() { return wait_bar(pfull(sub), np++ & 1, abort_word); };
            // a segment without this sub-tile: its buffers count as read once they are filled
            auto pass_k = [&](uint32_t tile) -> bool {
                if (!wait_k(tile)) return false;
                if (lane == 0) arrive(kempty(tile & 1));
                return true;
            };
            auto pass_v = [&](uint32_t tile) -> bool {
                if (!wait_v(tile)) return false;
                if (lane == 0) arrive(vempty(tile & 1));
                return true;
            };
            Segment seg;
            bool more = next_seg(seg);
            while (run && more) {
                const int n = __shfl_sync(ALL, seg.tb - seg.pl.tile, 0);
                const bool takes = __shfl_sync(ALL, sub == 0 || seg.rows - seg.pl.r0 > 128, 0);
                // S of the first key tile (P V of the segment before is on its way)
                if (takes) {
                    run = wait_q() && wait_k(nk) && lock();
                    if (!run) break;
                    tc::fence_after();
                    issue_s(nk);
                } else if (!(run = pass_k(nk))) {
                    break;
                }
                for (int j = 0; run && j < n - 1; ++j, ++nk) {
                    if (takes) {
                        run = wait_v(nk) && wait_k(nk + 1) && wait_p() && lock();
                        if (!run) break;
                        tc::fence_after();
                        issue_o(nk, j == 0);
                        issue_s(nk + 1);
                    } else {
                        run = pass_v(nk) && pass_k(nk + 1);
                    }
                }
                if (!run) break;
                if (takes) {
                    run = wait_v(nk) && wait_p() && lock();
                    if (!run) break;
                    tc::fence_after();
                    issue_o(nk, n == 1);
                    __syncwarp();
                    if (lane == 0) unlock();
                } else if (!(run = pass_v(nk))) {
                    break;
                }
                ++nk;
                more = next_seg(seg);
            }
            if (tc::elect_one()) tc::commit(drain);                           // products still in flight end before the tensor memory is given back
        }
        __syncwarp();
    } else if (warp >= kSoftWarps) {
        // ---- codes -> f16 tiles.  A warp takes 32 keys of a tile; lane = (row of
        // 8, 16-byte chunk), so a quarter-warp's stores fill a core matrix.
        // Scales go to a ring of kMetas: tile j + 4's are written once V of tile j + 3
        // is, for which P V of tile j + 1 had to be done, so both softmaxes are past
        // tile j and its slot is free.
        fewer_regs<Regs<FP4>::CONV>();
        constexpr int CH = D / 64, N = 4 * CH;           // 64-byte column groups, 16-byte pieces per thread and operand
        const int cw = warp - kSoftWarps, row = lane & 7, chunk = lane >> 3;
        uint32_t nt = 0;
        Segment ahead;
        int tile_ahead = 0;
        bool have = next_seg(ahead);
        // lane = (tile lane / 2, 16-key group lane % 2) of 16 tiles: its first row among the cache's (-1: not stored) and scales
        int64_t boff = -1;
        float bks = 0.0f, bvs = 0.0f, blg = 0.0f, brv = 0.0f;
        uint32_t bmiss = 0;
        int batch = -1, cur = 0;                         // first tile of the 16 (-1: none), the one to be stored next
        int64_t off[2] = {0, 0};
        int rows[2] = {0, 0};                            // stored rows of the two groups
        auto offsets = [&]() {
            if (batch < 0 || tile_ahead >= batch + 16) {
                batch = tile_ahead;
                const int key = ahead.key0() + (batch + (lane >> 1)) * kTcKeys + 32 * cw + 16 * (lane & 1);
                // groups that end before every row's window are not read: their blocks may be another request's by now
                const bool there = batch + (lane >> 1) < ahead.tb && key < ahead.rq.kv && key + 16 > ahead.low;
                const int32_t blk = there ? a.table[ahead.b * a.table_stride + key / a.S] : -1;
                const bool ok = blk >= 0 && blk < a.n_blocks;
                if (there && !ok) flag_error(a.err_flag, CSA2_FLAG_BAD_INDEX);
                const int64_t bh = ok ? (int64_t)blk * a.Hkv + ahead.pl.h : 0;
                boff = ok ? bh * a.S + (key & (a.S - 1)) : -1;
                if constexpr (!FP4) {
                    bks = ok ? a.k_scale[bh] : 0.0f;
                    bvs = ok ? a.v_scale[bh] : 0.0f;
                    blg = log_scale(bvs);
                    brv = rcp(bvs) * kDownFactor;
                }
                bmiss = __ballot_sync(ALL, !ok);
            }
            cur = tile_ahead - batch;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t at = __shfl_sync(ALL, boff, 2 * cur + u);
                const int left = ahead.rq.kv - (ahead.key0() + tile_ahead * kTcKeys + 32 * cw + 16 * u);
                rows[u] = at < 0 ? 0 : min(left, 16);
                off[u] = at < 0 ? 0 : at * (FP4 ? 1 : D);
            }
        };
        // The next tile's rows travel into the warp's own part of shared memory
        // (registers would do, but the softmax has them): whole rows per copy, chunks
        // swizzled, so that copies touch full lines and the reads below every bank.
        const uint32_t stage_k = sb + L::OFF_STAGE + cw * 32 * D, stage_v = stage_k + L::KV / 2;
        // Half as many bytes, the 4-bit cache's codes stay in registers: the products are
        // near what shared memory can feed them, and staging would ask it for a tenth more.
        // A lane holds, of every piece of 32 channels that it converts (row of 8, piece; of 64
        // channels every other 8 rows), the codes and the two scales.
        constexpr int PIECES = D / 32, STEP = 4 / PIECES, HELD = 4 / STEP;
        struct Held {
            uint4 c[HELD];
            uint32_t sc[HELD];
        } held_k, held_v;
        const int piece = chunk % PIECES, g0 = chunk / PIECES;
        auto hold = [&](Held &x, const uint8_t *codes, const uint8_t *scales) {
            if (have) {
#pragma unroll
                for (int i = 0; i < HELD; ++i) {
                    const int r = 8 * (i * STEP + g0) + row;                 // of the warp's 32
                    const bool there = (r & 15) < (r >> 4 ? rows[1] : rows[0]);      // rows that are not there read as zero
                    const int64_t at = (r >> 4 ? off[1] : off[0]) + (r & 15);
                    x.c[i] = there ? *reinterpret_cast<const uint4 *>(codes + at * (D / 2) + 16 * piece) : make_uint4(0, 0, 0, 0);
                    x.sc[i] = there ? *reinterpret_cast<const uint16_t *>(scales + at * (D / 16) + 2 * piece) : 0;
                }
            }
        };
        auto convert = [&](uint32_t dst, const Held &x) {
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                const uint32_t to = dst + (4 * cw + i * STEP + g0) * L::GROUP + 4 * piece * 128 + row * 16;
                const uint32_t w[4] = {x.c[i].x, x.c[i].y, x.c[i].z, x.c[i].w}, sc = e4m3x2_to_f16x2(x.sc[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t h[4];
                    e2m1x8_to_f16(w[k], __byte_perm(sc, 0, k < 2 ? 0x1010 : 0x3232), h);
                    sts128(to + k * 128, h[0], h[1], h[2], h[3]);
                }
            }
        };
        auto fetch = [&](uint32_t stage, const uint8_t *codes) {
            if (have) {
                constexpr int CPR = D / 16, RPI = 32 / CPR;                  // chunks per row, rows per copy
                const int c = lane % CPR, r0 = lane / CPR;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int u = i / (N / 2), r = (i % (N / 2)) * RPI + r0; // 16-key group, row of it
                    const bool there = r < rows[u];                          // rows that are not there read as zero
                    cp_async16(stage + chunk_at<D>(16 * u + r, c), there ? (const void *)(codes + off[u] + r * D + 16 * c) : a.q, there ? 16 : 0);
                }
            }
            cp_async_commit();
        };
        auto store = [&](uint32_t dst, uint32_t stage) {
            cp_async_wait<1>();                          // all but the newest of the copies
            __syncwarp();
            uint4 c[N];
#pragma unroll
            for (int i = 0; i < N; ++i) c[i] = lds128(stage + chunk_at<D>(8 * (i / CH) + row, 4 * (i % CH) + chunk));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int g = i / CH;
                const uint32_t to = dst + (4 * cw + g) * L::GROUP + (8 * (i % CH) + 2 * chunk) * 128 + row * 16;
                uint32_t h[8];
                e4m3x4_to_f16x2x2(c[i].x, h[0], h[1]);
                e4m3x4_to_f16x2x2(c[i].y, h[2], h[3]);
                e4m3x4_to_f16x2x2(c[i].z, h[4], h[5]);
                e4m3x4_to_f16x2x2(c[i].w, h[6], h[7]);
                sts128(to, h[0], h[1], h[2], h[3]);
                sts128(to + 128, h[4], h[5], h[6], h[7]);
            }
        };
        tile_ahead = ahead.pl.tile;
        bool loaded = false;                             // tile nt is on its way
        while (loaded || have) {
            const int buf = nt & 1;
            const uint32_t par = ((nt >> 1) & 1) ^ 1;
            if (loaded) {
                TileMeta &m = metas[nt % kMetas];
                if ((lane >> 1) == cur) {                // the lanes with the tile's scales
                    const int u = 2 * cw + (lane & 1);
                    if constexpr (!FP4) m.ks[u] = bks, m.vs[u] = bvs, m.lg[u] = blg, m.rv[u] = brv;
                    if (!(lane & 1)) m.missing[cw] = ((bmiss >> lane) & 3) << (2 * cw);
                }
                __syncwarp();
                if (lane == 0) arrive(mfull(nt % kMetas));
            }
            if (have) offsets();
            if (loaded) {
                if (!wait_bar(kempty(buf), par, abort_word)) break;
                if constexpr (FP4) convert(sb + L::OFF_K + buf * L::KV, held_k);
                else store(sb + L::OFF_K + buf * L::KV, stage_k);
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive(kfull(buf));
            }
            if constexpr (FP4) hold(held_k, a.k_codes, a.k_scale4);
            else fetch(stage_k, a.k_codes);
            if (loaded) {
                if (!wait_bar(vempty(buf), par, abort_word)) break;
                if constexpr (FP4) convert(sb + L::OFF_V + buf * L::KV, held_v);
                else store(sb + L::OFF_V + buf * L::KV, stage_v);
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive(vfull(buf));
                ++nt;
            }
            loaded = have;
            if constexpr (FP4) hold(held_v, a.v_codes, a.v_scale4);
            else fetch(stage_v, a.v_codes);
            if (have) {
                if (++tile_ahead >= ahead.tb) {          // the tile after the one that travels
                    have = next_seg(ahead);
                    tile_ahead = ahead.pl.tile;
                    batch = -1;
                }
            }
        }
    } else {
        more_regs<Regs<FP4>::SOFT>();
        // ---- softmax: thread = row
        const int sub = warp >> 2, rr = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + L::COL_S + sub * 128, to = tmem + lanes + L::COL_O + sub * D;
        uint32_t nt = 0, ns = 0;                         // key tiles of the CTA so far; of this sub-tile
        Segment seg;
        float zf = 0.0f;
        // The warp's 32 rows of Q into shared memory; zf: the logit factor of this
        // thread's row.  A copy takes 64 bytes of 8 rows (lane % 8 the row), so that a
        // quarter-warp's pieces fill a core matrix; each lane then scales the pieces
        // that it has copied, in place.  Rolled loops: the code is wanted once per
        // segment, and fetching its instructions is what it would wait for.
        auto load_q = [&](const Segment &s) {
            constexpr int CH = D / 32;                   // 16-byte pieces of a row per lane
            const int r8 = lane & 7, c4 = lane >> 3, w0 = s.pl.r0 + 128 * sub + 32 * (warp & 3);
            const uint32_t dst = sb + L::OFF_Q + sub * L::Q + 4 * (warp & 3) * L::GROUP + c4 * 128 + r8 * 16;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int row = w0 + 8 * i + r8;
                const bool real = row < s.rows;
                const int tok = real ? row / a.G : 0, hq = s.pl.h * a.G + (real ? row - tok * a.G : 0);
                const uint16_t *src = a.q + (s.rq.row0 + tok) * a.q_token_stride + hq * a.q_head_stride + 8 * c4;
#pragma unroll
                for (int c = 0; c < CH; ++c)             // rows that are not there are zero
                    cp_async16(dst + i * L::GROUP + c * 512, real ? (const void *)(src + 32 * c) : a.q, real ? 16 : 0);
            }
            cp_async_commit();
            cp_async_wait<0>();
            const float sign = a.logit_scale < 0.0f ? -1.0f : 1.0f;      // goes to q: factors are not negative
            if (HALF) zf = fabsf(a.logit_scale);
            if (!HALF || a.logit_scale < 0.0f) {
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint4 v[CH];
                    float top = 0.0f, mul = sign;
#pragma unroll
                    for (int c = 0; c < CH; ++c) v[c] = lds128(dst + i * L::GROUP + c * 512);
                    if (!HALF) {
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float2 f = unpack_in<HALF>(w[x]);
                                top = max3(top, fabsf(f.x), fabsf(f.y));
                            }
                        }
                        top = fmaxf(top, __shfl_xor_sync(ALL, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(ALL, top, 16));
                        // largest magnitude to [2^14, 2^15); a row below 2^-100 keeps that factor
                        const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
                        mul = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
                        if (i == c4) zf = fabsf(a.logit_scale) / mul;    // row 8 i + r8 is this thread's
                        mul *= sign;
                    }
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float2 f = unpack_in<HALF>(w[x]);
                            w[x] = pack_f16(f.x * mul, f.y * mul);
                        }
                        sts128(dst + i * L::GROUP + c * 512, w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if constexpr (TMEM_Q) {                      // this thread's row to its lane
                __syncwarp();
                const uint32_t src = sb + L::OFF_Q + sub * L::Q + (4 * (warp & 3) + c4) * L::GROUP + r8 * 16;
#pragma unroll
                for (int c = 0; c < D / 8; c += 4) {
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint4 v = lds128(src + (c + x) * 128);
                        w[4 * x] = v.x, w[4 * x + 1] = v.y, w[4 * x + 2] = v.z, w[4 * x + 3] = v.w;
                    }
                    tc::tmem_st16(tmem + lanes + L::COL_Q + sub * (D / 2) + 4 * c, w);
                }
                tc::tmem_st_wait();
                tc::fence_before();
            } else {
                tc::fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) arrive(qfull(sub));
        };
        int row = 0, n = 0;                              // this thread's row, the segment's key tiles
        bool busy = false, real = false, whole = false, first_part = false;
        int64_t o_row = 0;
        float M = NEG_INF, MV = NEG_INF, l = 0.0f;
        for (;;) {
            Segment nxt;
            const bool more = next_seg(nxt);
            const bool takes = more && (sub == 0 || nxt.rows - nxt.pl.r0 > 128);
            if (takes) load_q(nxt);                      // Q is free: S of the last tile is done
            if (busy) {                                  // O of the segment before
                if (!wait_bar(ofull(sub), (ns - 1) & 1, abort_word)) break;
                tc::fence_after();
                if (FP4) MV = M;
                const float ref = M == NEG_INF ? 0.0f : M, refv = MV == NEG_INF ? 0.0f : MV;
                const float scale = exp2f(refv - ref), inv = l > 0.0f ? kDownFactor / l : (l == 0.0f ? 0.0f : l);
                float *part = a.partial_tc + ((2 * (int64_t)blockIdx.x + first_part) * kTcRows + 128 * sub + rr) * (D + 4);
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[32];
                    __syncwarp();
                    tc::tmem_ld32(to + 32 * c, r);
                    tc::tmem_ld_wait();
                    if (whole) {
                        // four lanes exchange their four 16-byte pieces, so that a store takes 64 bytes of 8 rows
                        uint32_t w[4][4];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i / 4][i % 4] = pack_out<HALF>(__uint_as_float(r[2 * i]) * inv * scale, __uint_as_float(r[2 * i + 1]) * inv * scale);
#pragma unroll
                        for (int d = 1; d < 4; d *= 2)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                if (x & d) continue;
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const bool up = lane & d;
                                    const uint32_t got = __shfl_xor_sync(ALL, up ? w[x][y] : w[x + d][y], d);
                                    (up ? w[x][y] : w[x + d][y]) = got;
                                }
                            }
                        // piece x is now row (lane & ~3) + x's, its 16 bytes at lane % 4
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int64_t o = __shfl_sync(ALL, o_row, (lane & ~3) + x);
                            if (__shfl_sync(ALL, (int)real, (lane & ~3) + x))
                                *reinterpret_cast<uint4 *>(a.out + o * D + 32 * c + 8 * (lane & 3)) = make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
                        }
                    } else if (real) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<uint4 *>(part + 32 * c + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
                    }
                }
                __syncwarp();
                tc::fence_before();
                if (real && whole && a.lse)
                    a.lse[o_row] = l > 0.0f || l != l ? (M + log2f(l)) * 0.69314718055994531f : NEG_INF;
                if (real && !whole) *reinterpret_cast<float4 *>(part + D) = make_float4(M, MV, l, 0.0f);
            }
            if (!more) break;
            seg = nxt;
            n = seg.tb - seg.pl.tile;
            busy = takes;
            if (!busy) {
                nt += n;
                continue;
            }
            row = seg.pl.r0 + 128 * sub + rr;
            real = row < seg.rows;
            const int tok = real ? row / a.G : 0;
            o_row = (seg.rq.row0 + tok) * a.Hq + seg.pl.h * a.G + (row - tok * a.G);
            whole = seg.pl.tile == 0 && seg.tb == seg.pl.tiles;
            first_part = seg.pl.tile == 0;
            // rows that are not there see everything: they hold no warp back, and are not stored
            const int pos = real ? max(-1, seg.rq.kv - seg.rq.n + tok) : 0x7FFFFFF0;
            const int first = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
            M = MV = NEG_INF;
            l = 0.0f;
            for (int j = 0; j < n; ++j, ++nt, ++ns) {
                const TileMeta &m = metas[nt % kMetas];
                const int key0 = seg.key0() + (seg.pl.tile + j) * kTcKeys;
                const int lo = max(first - key0, 0), hi = min(pos + 1 - key0, kTcKeys);
                // The common case, one exponential and no maximum: with the references as
                // they are, P = 2^(s f + log2(2^kUp vs) - Mv), and l gains sum P / (2^kUp vs) 2^(Mv - M).
                // Where the sum of a row's P shows that one may leave f16, Mv is raised by a
                // whole power of two and P computed once more; a scale so far from the others
                // that P would not carry its keys' part of l takes the way with maxima.
                // P goes to TMEM when that is known.  What depends on the scales
                // alone is settled before the scores arrive.  But a segment's first scores
                // come first: a sub-tile that had no part in the last segment may be here
                // several tiles early, while the barrier of the scales' slot still counts an
                // older round.  From the second tile on, S of the tile before says that the
                // scales of all rounds before have arrived.
                auto wait_s = [&]() { return wait_bar(sfull(sub), ns & 1, abort_word); };
                if (j == 0 && !(run = wait_s())) break;
                if (!(run = wait_bar(mfull(nt % kMetas), (nt / kMetas) & 1, abort_word))) break;
                const uint32_t missing = m.missing[0] | m.missing[1] | m.missing[2] | m.missing[3];
                const bool mask = lo > 0 || hi < kTcKeys || missing != 0;
                bool fast;
                if constexpr (FP4) {
                    fast = __all_sync(ALL, !mask && M > NEG_INF);
                } else {
                    const float4 lg0 = *reinterpret_cast<const float4 *>(m.lg), lg1 = *reinterpret_cast<const float4 *>(m.lg + 4);
                    const float least = fminf(fminf(fminf(lg0.x, lg0.y), fminf(lg0.z, lg0.w)), fminf(fminf(lg1.x, lg1.y), fminf(lg1.z, lg1.w)));
                    const float most = fmaxf(fmaxf(fmaxf(lg0.x, lg0.y), fmaxf(lg0.z, lg0.w)), fmaxf(fmaxf(lg1.x, lg1.y), fmaxf(lg1.z, lg1.w)));
                    fast = __all_sync(ALL, !mask && M - MV + least > -kSpread && M - MV + most < kSpread);
                }
                if (j > 0 && !(run = wait_s())) break;
                tc::fence_after();
                // scores of the keys 32 c .. 32 c + 31 that the row does not see: -inf
                auto hide = [&](int c, uint32_t (&r)[32]) {
                    const int l0 = max(lo - 32 * c, 0), h0 = min(hi - 32 * c, 32);
                    uint32_t seen = h0 <= 0 || l0 >= 32 ? 0u : (0xFFFFFFFFu >> (32 - h0)) & (0xFFFFFFFFu << l0);
                    if ((missing >> (2 * c)) & 1) seen &= 0xFFFF0000u;
                    if ((missing >> (2 * c)) & 2) seen &= 0x0000FFFFu;
                    if (__all_sync(ALL, seen == 0xFFFFFFFFu)) return;    // of a tile on the diagonal mostly two or three quarters
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((seen >> i) & 1)) r[i] = 0xff800000u;
                };
                // O so far to another reference; S followed the products that it waited for
                auto rescale = [&](float by) {
#pragma unroll 1
                    for (int x = 0; x < D; x += 32) {
                        uint32_t r[32];
                        tc::tmem_ld32(to + x, r);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t o[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(r[16 * c + i]) * by);
                            tc::tmem_st16(to + x + 16 * c, o);
                        }
                    }
                };
                if constexpr (FP4) {
                    // No scales between scores and weights: one reference, P = 2^(s f + kUp - M).
                    const float f = fmaxf(zf, 1e-38f);       // not 0, so that a hidden score of -inf stays -inf
                    const uint64_t ff = f2(f, f);
                    for (bool raised = false; fast; raised = true) {
                        const float at = kUp - M;
                        const uint64_t aa = f2(at, at);
                        uint64_t sum0 = f2(0.0f, 0.0f), sum1 = sum0;
                        // 16 scores at a time, their sums and halves behind the exponentials of the next
                        uint32_t p[4][16], r[2][32];
                        float e[2][16];
                        auto take = [&](int g) {
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float e0 = e[g & 1][i], e1 = e[g & 1][i + 1];
                                if (i & 2) sum1 = add2(sum1, f2(e0, e1));
                                else sum0 = add2(sum0, f2(e0, e1));
                                p[g / 2][8 * (g & 1) + i / 2] = pack_f16(e0, e1);
                            }
                        };
                        tc::tmem_ld32(ts, r[0]);
#pragma unroll
                        for (int g = 0; g < 8; ++g) {
                            const int c = g / 2, at16 = 16 * (g & 1);
                            if (at16 == 0) {
                                tc::tmem_ld_wait();
                                if (c < 3) tc::tmem_ld32(ts + 32 * (c + 1), r[(c + 1) & 1]);
                            }
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float2 z = un2(fma2(f2u(r[c & 1][at16 + i], r[c & 1][at16 + i + 1]), ff, aa));
                                e[g & 1][i] = ex2(z.x), e[g & 1][i + 1] = ex2(z.y);
                            }
                            if (g) take(g - 1);
                        }
                        take(7);
                        const float2 x = un2(add2(sum0, sum1));
                        const float total = x.x + x.y;
                        if (__all_sync(ALL, total < kMostP)) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) tc::tmem_st16(ts + 16 * c, p[c]);
                            l = fmaf(total, kDownFactor, l);
                            break;
                        }
                        // once: of scores beyond 2^24 a higher M may round to the same, or further up
                        fast = !raised && __all_sync(ALL, total < kMostRaise);
                        if (fast) {                          // all 32 rows' sums to 2^kUp, as far as they exceed it
                            const float m1 = M + max(0, (int)(__float_as_uint(total) >> 23) - 127 - kUp), by = ex2(M - m1);
                            rescale(by);
                            l *= by;
                            M = m1;
                        }
                    }
                    if (!fast) {
                        const bool masked = __any_sync(ALL, mask);
                        uint32_t r[2][32];
                        float tz = NEG_INF;
#pragma unroll 1
                        for (int c = 0; c < 4; c += 2) {
                            tc::tmem_ld32(ts + 32 * c, r[0]);
                            tc::tmem_ld32(ts + 32 * c + 32, r[1]);
                            tc::tmem_ld_wait();
                            if (masked) hide(c, r[0]), hide(c + 1, r[1]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float t0 = __uint_as_float(r[k][0]), t1 = __uint_as_float(r[k][1]);
#pragma unroll
                                for (int i = 2; i < 30; i += 4) {
                                    t0 = max3(t0, __uint_as_float(r[k][i]), __uint_as_float(r[k][i + 1]));
                                    t1 = max3(t1, __uint_as_float(r[k][i + 2]), __uint_as_float(r[k][i + 3]));
                                }
                                tz = fmaxf(tz, fmaxf(max3(t0, t1, __uint_as_float(r[k][30])), __uint_as_float(r[k][31])));
                            }
                        }
                        tz = __fmul_rn(tz, f);
                        // The references move when a row's scores exceed one by more than the slack, or at a row's
                        // first key; then those of all 32 rows do, as far as they are exceeded, so that the next
                        // tiles are the less likely to need it.
                        const bool up = __any_sync(ALL, tz - M > kSlack) && tz > M;
                        const float grow = up ? ex2(M - tz) : 1.0f;
                        l *= grow;
                        if (up) M = tz;
                        if (j > 0 && __any_sync(ALL, up)) rescale(grow);
                        const float ref = M == NEG_INF ? 0.0f : M;
                        uint64_t sum = f2(0.0f, 0.0f);
#pragma unroll 1
                        for (int c = 0; c < 4; c += 2) {
                            tc::tmem_ld32(ts + 32 * c, r[0]);
                            tc::tmem_ld32(ts + 32 * c + 32, r[1]);
                            tc::tmem_ld_wait();
                            if (masked) hide(c, r[0]), hide(c + 1, r[1]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint32_t p[16];
#pragma unroll
                                for (int i = 0; i < 32; i += 2) {
                                    // rounded as the maximum was, before the reference is taken off, so that none is beyond it
                                    const float z0 = __fmul_rn(__uint_as_float(r[k][i]), f), z1 = __fmul_rn(__uint_as_float(r[k][i + 1]), f);
                                    const float e0 = ex2(__fadd_rn(z0, -ref) + kUp), e1 = ex2(__fadd_rn(z1, -ref) + kUp);
                                    sum = add2(sum, f2(e0, e1));
                                    p[i / 2] = pack_f16(e0, e1);
                                }
                                tc::tmem_st16(ts + 16 * (c + k), p);
                            }
                        }
                        const float2 s2 = un2(sum);
                        l = fmaf(s2.x + s2.y, kDownFactor, l);
                    }
                } else {
                    for (bool raised = false; fast; raised = true) {
                        const float back = ex2(MV - M);
                        uint32_t p[4][16];
                        float gain = 0.0f, total = 0.0f;
                        uint32_t r[2][32];
                        tc::tmem_ld32(ts, r[0]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tc::tmem_ld_wait();
                            if (c < 3) tc::tmem_ld32(ts + 32 * (c + 1), r[(c + 1) & 1]);
                            const float2 ks = *reinterpret_cast<const float2 *>(&m.ks[2 * c]), lg = *reinterpret_cast<const float2 *>(&m.lg[2 * c]),
                                         rv = *reinterpret_cast<const float2 *>(&m.rv[2 * c]);
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                const float f = factor(zf, g ? ks.y : ks.x), at = (g ? lg.y : lg.x) - MV;
                                const uint64_t ff = f2(f, f), aa = f2(at, at);
                                uint64_t sum0 = f2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    const float2 z = un2(fma2(f2u(r[c & 1][16 * g + i], r[c & 1][16 * g + i + 1]), ff, aa));
                                    const float e0 = ex2(z.x), e1 = ex2(z.y);
                                    if (i & 2) sum1 = add2(sum1, f2(e0, e1));
                                    else sum0 = add2(sum0, f2(e0, e1));
                                    p[c][8 * g + i / 2] = pack_f16(e0, e1);
                                }
                                const float2 x = un2(add2(sum0, sum1));
                                const float y = x.x + x.y;
                                total += y;
                                gain += y * (g ? rv.y : rv.x);
                            }
                        }
                        if (__all_sync(ALL, total < kMostP && gain * back < kMostL)) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) tc::tmem_st16(ts + 16 * c, p[c]);
                            l += gain * back;
                            break;
                        }
                        // once: of scores beyond 2^24 a higher Mv may round to the same, or further up
                        fast = !raised && __all_sync(ALL, total < kMostRaise && gain * back < kMostL);
                        if (fast) {                          // all 32 rows' sums to 2^kUp, as far as they exceed it
                            const float mv1 = MV + max(0, (int)(__float_as_uint(total) >> 23) - 127 - kUp);
                            rescale(ex2(MV - mv1));
                            MV = mv1;
                        }
                    }
                    if (!fast) {
                        const bool masked = __any_sync(ALL, mask);
                        // 64 scores at a time, read again for P: all 128 do not fit beside the rest
                        uint32_t r[2][32];
                        float tz = NEG_INF, tv = NEG_INF;
#pragma unroll 1
                        for (int c = 0; c < 4; c += 2) {
                            tc::tmem_ld32(ts + 32 * c, r[0]);
                            tc::tmem_ld32(ts + 32 * c + 32, r[1]);
                            tc::tmem_ld_wait();
                            if (masked) hide(c, r[0]), hide(c + 1, r[1]);
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const uint32_t (&x)[32] = r[g / 2];
                                const int i0 = 16 * (g & 1);
                                float t0 = __uint_as_float(x[i0]), t1 = __uint_as_float(x[i0 + 1]);
#pragma unroll
                                for (int i = 2; i < 14; i += 4) {
                                    t0 = max3(t0, __uint_as_float(x[i0 + i]), __uint_as_float(x[i0 + i + 1]));
                                    t1 = max3(t1, __uint_as_float(x[i0 + i + 2]), __uint_as_float(x[i0 + i + 3]));
                                }
                                const float t = fmaxf(max3(t0, t1, __uint_as_float(x[i0 + 14])), __uint_as_float(x[i0 + 15])) * factor(zf, m.ks[2 * c + g]);
                                tz = fmaxf(tz, t);
                                tv = fmaxf(tv, t + (float)((int)((__float_as_uint(m.vs[2 * c + g]) >> 23) & 0xFFu) - 127));
                            }
                        }
                        // The references move when a row's scores exceed one by more than the slack, or at a row's
                        // first key; then those of all 32 rows do, as far as they are exceeded, so that the next
                        // tiles are the less likely to need it.
                        const bool due = tz - M > kSlack || tv - MV > kSlack;
                        const bool all = __any_sync(ALL, due), up = all && tz > M, upv = all && tv > MV;
                        if (up) {
                            l *= ex2(M - tz);
                            M = tz;
                        }
                        const float grow = upv ? ex2(MV - tv) : 1.0f;
                        if (upv) MV = tv;
                        if (j > 0 && __any_sync(ALL, upv)) rescale(grow);
                        const float ref = M == NEG_INF ? 0.0f : M, g2 = ex2(0.5f * (ref - (MV == NEG_INF ? 0.0f : MV)));     // 2^(M - Mv) in two steps
                        uint64_t sum = f2(0.0f, 0.0f);
#pragma unroll 1
                        for (int c = 0; c < 4; c += 2) {
                            tc::tmem_ld32(ts + 32 * c, r[0]);
                            tc::tmem_ld32(ts + 32 * c + 32, r[1]);
                            tc::tmem_ld_wait();
                            if (masked) hide(c, r[0]), hide(c + 1, r[1]);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint32_t p[16];
#pragma unroll
                                for (int g = 0; g < 2; ++g) {
                                    const float f = factor(zf, m.ks[2 * c + 2 * k + g]), w = fminf(m.vs[2 * c + 2 * k + g] * g2 * g2, kMostWeight) * kUpFactor;
                                    const uint64_t ww = f2(w, w);
#pragma unroll
                                    for (int i = 0; i < 16; i += 2) {
                                        // rounded as the maxima were, before the reference is taken off, so that none is beyond
                                        // them (a packed product and sum would be joined again, without that rounding)
                                        const float z0 = __fmul_rn(__uint_as_float(r[k][16 * g + i]), f), z1 = __fmul_rn(__uint_as_float(r[k][16 * g + i + 1]), f);
                                        const uint64_t e = f2(ex2(__fadd_rn(z0, -ref)), ex2(__fadd_rn(z1, -ref)));
                                        sum = add2(sum, e);
                                        const float2 x = un2(mul2(e, ww));
                                        p[8 * g + i / 2] = pack_f16(x.x, x.y);
                                    }
                                }
                                tc::tmem_st16(ts + 16 * (c + k), p);
                            }
                        }
                        const float2 s2 = un2(sum);
                        l += s2.x + s2.y;
                    }
                }
                tc::tmem_st_wait();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) arrive(pfull(sub));
            }
            if (!run) break;
        }
    }
    if (warp >= kMmaWarp && warp < kMmaWarp + 2) tc::mbar_wait(drain, 0, 1u << 20);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (tid == 0 && *abort_word) flag_error(a.err_flag, CSA2_FLAG_TIMEOUT);
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int D, bool HALF, bool FP4>
cudaError_t go(const PagedAttnArgs &a, cudaStream_t stream) {
    static bool done[64];
    cudaError_t e = ensure_smem_limit((const void *)paged_attn_tc_kernel<D, HALF, FP4>, Lay<D>::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn_tc_kernel<D, HALF, FP4>, dim3(paged_attn_tc_ctas()), dim3(kTcThreads), Lay<D>::SMEM, stream, a);
}

template <bool FP4>
cudaError_t go_for(const PagedAttnArgs &a, int D, bool half, cudaStream_t stream) {
    if (half) return D == 64 ? go<64, true, FP4>(a, stream) : go<128, true, FP4>(a, stream);
    return D == 64 ? go<64, false, FP4>(a, stream) : go<128, false, FP4>(a, stream);
}

}  // namespace

int paged_attn_tc_ctas() { return num_sms(); }

cudaError_t launch_paged_attn_tc(const PagedAttnArgs &a, int D, bool half, bool fp4, cudaStream_t stream) {
    return fp4 ? go_for<true>(a, D, half, stream) : go_for<false>(a, D, half, stream);
}

}  // namespace csa2
