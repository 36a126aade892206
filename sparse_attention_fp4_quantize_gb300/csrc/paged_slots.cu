// csa2_build_slots: block tables and slot maps of a ragged batch from the
// requests' lengths.
//
// With S tokens per block, held_b = ceil(kv_b / S) and after_b =
// ceil((kv_b + n_b) / S), everything a step needs is three prefix sums over the
// requests:
//   cu_b   = sum_{i<b} max(n_i, 0)             first row of request b
//   a_b    = sum_{i<b} (after_i - held_i)      first block it takes (those that fit)
//   f_b    = sum_{i<b, ended} held_i           where its blocks land on the free list
// A block index is then looked up, not searched for in order: block a of the
// step is entry size - 1 - a of the stack (free list, then freed blocks), and
// entry n_free + k of that stack is block k - f_b of the ended request b that
// holds k, found by bisection in f.
//
// One launch: every CTA computes the prefix sums of all requests itself (a few KB
// from L2, so no CTA waits for another's sums), then the CTAs share the rows, four
// per thread and step.  Where the results go to the inputs themselves (a captured
// step), the CTAs are one thread-block cluster and write them behind its barrier,
// when every CTA has read what they replace.
//
// Bound by latency: a launch, two loads in a row, three prefix sums, a bisection
// and a load.  On the GPU, from a cold L2: 32 requests decoding 7.7 us, 512 mixed
// (16384 rows, blocks of 16, some ended) 12.1 us, 2000 prompts (65536 rows) 10.3 us;
// a call from Python takes about 9 us of host time, so that only the last two show.
// With one cluster for every call the prompts took 16 us: eight CTAs have 13 rows
// per thread.
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace csa2 {
namespace {

constexpr int kMaxRequests = 8192;

struct SlotArgs {
    int B, M, S;
    int64_t table_stride, T, free_cap;
    const int32_t *kv_len, *new_len;
    int32_t *table, *free_list;
    const int32_t *free_count;
    int32_t *kv_out, *free_out, *cu, *positions;
    int64_t *slots;
    uint32_t *err_flag;
    bool wide;                       // slots and positions are 16-byte aligned
    bool in_place;                   // the CTAs are a cluster
};

// Exclusive prefix sums over the block of N values per thread; totals to all.
template <int N>
__device__ __forceinline__ void block_scan(int64_t (&v)[N], int64_t (*warp_sums)[32], int64_t (&total)[N]) {
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t s[N], w[N];
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] = v[n];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int64_t y = __shfl_up_sync(ALL, s[n], o);
            if (lane >= o) s[n] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int n = 0; n < N; ++n) warp_sums[n][warp] = s[n];
    __syncthreads();
    // every warp scans the warps' sums by itself
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = lane < warps ? warp_sums[n][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int64_t y = __shfl_up_sync(ALL, w[n], o);
            if (lane >= o) w[n] += y;
        }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        total[n] = __shfl_sync(ALL, w[n], 31);
        const int64_t before = __shfl_sync(ALL, w[n], warp - 1);     // of lane 31 for warp 0, not used
        v[n] = (warp ? before : 0) + s[n] - v[n];
    }
}

// Last b with a[b] <= x, of the nondecreasing a[0..n), a[0] <= x.
__device__ __forceinline__ int last_at_most(const int32_t *a, int n, int32_t x) {
    int lo = 0, hi = n;   // a[lo] <= x, and a[hi] > x or hi == n
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void build_slots_kernel(SlotArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int64_t warp_sums[3][32];
    __shared__ int32_t s_taken;
    int32_t *s_cu = sm;                    // first row
    int32_t *s_kv = s_cu + a.B;            // tokens held
    int32_t *s_take = s_kv + a.B;          // first block taken, -1: waits
    int32_t *s_freed = s_take + a.B;       // first place among the freed blocks
    const int rank = blockIdx.x, ranks = gridDim.x;
    const int tid = threadIdx.x, nt = blockDim.x;
    const uint32_t S = a.S;
    const int per = (a.B + nt - 1) / nt, b0 = tid * per, b1 = min(a.B, b0 + per);
    const int64_t cap = (int64_t)a.M * a.S;
    uint32_t flags = 0;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) s_taken = 0;

    // rows and freed blocks; n is bounded by T + 1, which fits no budget
    int64_t rows = 0, freed = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t k = a.kv_len[b], n = a.new_len[b];
        const int32_t kv = (int32_t)(k < 0 ? 0 : (k > cap ? cap : k));
        if (kv != k) flags |= CSA2_FLAG_BAD_INDEX;
        s_kv[b] = kv;
        if (n > 0) rows += n < a.T + 1 ? n : a.T + 1;
        if (n < 0) freed += (kv + S - 1) / S;
    }
    const int64_t fc = *a.free_count;
    int64_t sums[2] = {rows, freed}, totals[2];
    block_scan<2>(sums, warp_sums, totals);
    int64_t cu = sums[0], fr = sums[1];
    const int64_t n_rows = totals[0], n_freed = totals[1];
    const int64_t n_free = fc < 0 ? 0 : (fc > a.free_cap ? a.free_cap : fc);
    if (fc != n_free) flags |= CSA2_FLAG_BAD_INDEX;
    const int64_t size = n_free + n_freed;

    int64_t need = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t n = a.new_len[b];
        const uint32_t kv = s_kv[b], held = (kv + S - 1) / S;
        s_cu[b] = (int32_t)(cu < a.T ? cu : a.T);
        s_freed[b] = (int32_t)fr;
        uint32_t more = 0;                 // blocks it asks for, if its tokens fit
        if (n > 0) {
            cu += n < a.T + 1 ? n : a.T + 1;
            if (cu <= a.T && kv + n <= cap) need += more = (kv + (uint32_t)n + S - 1) / S - held;
            else flags |= CSA2_FLAG_BAD_SLOT, more = 0xFFFFFFFFu;
        } else if (n < 0) {
            fr += held;
        }
        s_take[b] = (int32_t)more;
    }
    int64_t wanted[1] = {need}, n_need[1];
    block_scan<1>(wanted, warp_sums + 2, n_need);
    int64_t take = wanted[0];
    int taken = 0;
    for (int b = b0; b < b1; ++b) {
        const uint32_t more = (uint32_t)s_take[b];
        int32_t first = 0;
        if (more == 0xFFFFFFFFu) {
            first = -1;
        } else if (more) {
            if (take + more <= size) {
                first = (int32_t)take;
                taken = (int)(take + more);
            } else {
                first = -1;
                flags |= CSA2_FLAG_NO_BLOCKS;
            }
            take += more;
        }
        s_take[b] = first;
    }
    if (taken) atomicMax(&s_taken, taken);   // a maximum: the same in any order
    __syncthreads();
    int64_t count = size - s_taken;
    if (count > a.free_cap) {
        count = a.free_cap;
        flags |= CSA2_FLAG_BAD_INDEX;
    }

    auto freed_block = [&](int64_t k) -> int32_t {
        const int b = last_at_most(s_freed, a.B, (int32_t)k);
        return a.table[b * a.table_stride + (k - s_freed[b])];
    };
    // four rows per thread and step: one search, and mostly one block, for all of them
    const int64_t step = (int64_t)ranks * nt;
    const int64_t end = n_rows < a.T ? n_rows : a.T;
    for (int64_t t0 = ((int64_t)rank * nt + tid) * 4; t0 < a.T; t0 += step * 4) {
        int64_t slot[4];
        int32_t pos[4], b = 0, block = -1;
        uint32_t page = 0xFFFFFFFFu;                 // whose block is at hand
        if (t0 < end) b = last_at_most(s_cu, a.B, (int32_t)t0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + i;
            slot[i] = -1;
            pos[i] = -1;
            if (t >= end) continue;
            while (b + 1 < a.B && s_cu[b + 1] <= t) ++b, page = 0xFFFFFFFFu;
            const int32_t first = s_take[b];
            if (first < 0) continue;
            const uint32_t kv = s_kv[b], p = kv + (uint32_t)(t - s_cu[b]), now = p / S, row = p - now * S;
            if (now != page) {
                page = now;
                const uint32_t held = (kv + S - 1) / S;
                int32_t *entry = a.table + b * a.table_stride + page;
                if (page < held) {
                    block = *entry;
                } else {
                    const int64_t at = size - 1 - (first + (int64_t)(page - held));
                    block = at < n_free ? a.free_list[at] : freed_block(at - n_free);
                    if (row == 0) *entry = block;    // the block's first token is among the new ones
                }
            }
            pos[i] = (int32_t)p;
            if (block >= 0) slot[i] = (int64_t)block * S + row;
            else flags |= CSA2_FLAG_BAD_INDEX;
        }
        if (a.wide && t0 + 4 <= a.T) {
            reinterpret_cast<longlong2 *>(a.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
            reinterpret_cast<longlong2 *>(a.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
            if (a.positions) *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + i < a.T) {
                    a.slots[t0 + i] = slot[i];
                    if (a.positions) a.positions[t0 + i] = pos[i];
                }
        }
    }
    for (int64_t k = (int64_t)rank * nt + tid; k < count - n_free; k += step) a.free_list[n_free + k] = freed_block(k);
    if (flags) flag_error(a.err_flag, flags);

    if (a.in_place) cg::this_cluster().sync();   // every CTA has read kv_len and free_count
    if (rank == 0) {
        for (int b = tid; b < a.B; b += nt) {
            const int64_t n = a.new_len[b];
            const int32_t kv = s_kv[b];
            a.kv_out[b] = n < 0 ? 0 : (n > 0 && s_take[b] >= 0 ? (int32_t)(kv + n) : kv);
            a.cu[b] = s_cu[b];
        }
        if (tid == 0) {
            a.cu[a.B] = (int32_t)end;
            *a.free_out = (int32_t)count;
        }
    }
}

// Whether n words at p share one with the table's rows (B of M words, `stride` words apart).
bool rows_meet(const int32_t *table, int64_t B, int64_t M, int64_t stride, const void *p, int64_t n) {
    const int64_t x = (int64_t)((uintptr_t)p - (uintptr_t)table), end = x + 4 * n, pitch = 4 * stride;      // bytes from the table's begin
    if (n == 0 || end <= 0 || x / pitch >= B) return false;
    const int64_t row = x < 4 * M ? 0 : (x - 4 * M) / pitch + 1;           // the first row that ends behind x
    return row < B && row * pitch < end;
}

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" csa2_status csa2_build_slots(int B, int M, int64_t table_stride, int S, int64_t T, int64_t free_cap,
                                        const int32_t *kv_len, const int32_t *new_len, int32_t *block_table,
                                        int32_t *free_list, const int32_t *free_count, int32_t *kv_len_out,
                                        int32_t *free_count_out, int32_t *cu_len, int32_t *positions, int64_t *slots,
                                        uint32_t *err_flag, csa2_stream_t stream) {
    clear_error();
    CSA2_REQUIRE(B >= 1 && B <= kMaxRequests, "build_slots: B=%d not in [1, %d]", B, kMaxRequests);
    CSA2_REQUIRE(S >= 1 && M >= 1 && (int64_t)M * S < (1ll << 31), "build_slots: S=%d, M=%d: need M * S < 2^31", S, M);
    CSA2_REQUIRE((int64_t)B * M < (1ll << 31), "build_slots: B * M = %lld entries", (long long)B * M);
    CSA2_REQUIRE(table_stride >= M, "build_slots: table_stride=%lld < M=%d", (long long)table_stride, M);
    CSA2_REQUIRE(table_stride < (1ll << 40), "build_slots: table_stride=%lld", (long long)table_stride);
    CSA2_REQUIRE(T >= 0 && T <= (1ll << 30), "build_slots: T=%lld not in [0, 2^30]", (long long)T);
    CSA2_REQUIRE(free_cap >= 0 && free_cap < (1ll << 31), "build_slots: free_cap=%lld", (long long)free_cap);
    CSA2_REQUIRE(kv_len && new_len && block_table && free_count && kv_len_out && free_count_out && cu_len,
                 "build_slots: null pointer");
    CSA2_REQUIRE((free_list || free_cap == 0) && (slots || T == 0), "build_slots: null pointer");
    CSA2_REQUIRE(aligned(slots, 8), "build_slots: slots must be 8-byte aligned");
    for (const void *p : {(const void *)kv_len, (const void *)new_len, (const void *)block_table, (const void *)free_list,
                          (const void *)free_count, (const void *)kv_len_out, (const void *)free_count_out,
                          (const void *)cu_len, (const void *)positions, (const void *)err_flag})
        CSA2_REQUIRE(aligned(p, 4), "build_slots: int32 arguments must be 4-byte aligned");
    // The CTAs read and write side by side: only the lengths' and the count's outputs may take
    // the place of their inputs, all else stands apart.  Inputs first, then what is written.
    const bool in_place = kv_len_out == kv_len || free_count_out == free_count;
    const struct Span { const void *p; int64_t n; } span[10] = {           // 4-byte words
        {kv_len, B}, {free_count, 1}, {new_len, B}, {kv_len_out, B}, {free_count_out, 1}, {cu_len, B + 1ll},
        {positions, positions ? T : 0}, {slots, 2 * T}, {free_list, free_cap},
        {err_flag, err_flag != nullptr}};
    auto apart = [](const Span &x, const Span &y) {
        return !x.n || !y.n || (uintptr_t)x.p + 4 * x.n <= (uintptr_t)y.p || (uintptr_t)y.p + 4 * y.n <= (uintptr_t)x.p;
    };
    for (int i = 0; i < 10; ++i) {
        for (int o = i < 3 ? 3 : i + 1; o < 10; ++o) {
            const bool own = o == i + 3 && i < 2 && span[o].p == span[i].p;
            CSA2_REQUIRE(own || apart(span[i], span[o]), i < 3 ? "build_slots: an output overlaps an input"
                                                               : "build_slots: an output overlaps another");
        }
        CSA2_REQUIRE(!rows_meet(block_table, B, M, table_stride, span[i].p, span[i].n), "build_slots: block_table overlaps another tensor");
    }
    const SlotArgs args = {B, M, S, table_stride, T, free_cap, kv_len, new_len, block_table, free_list, free_count,
                           kv_len_out, free_count_out, cu_len, positions, slots, err_flag,
                           aligned(slots, 16) && aligned(positions, 16), in_place};
    const size_t smem = (size_t)B * 4 * sizeof(int32_t);
    static bool done[64];
    if (smem > 40 * 1024)
        CSA2_CUDA_CALL(ensure_smem_limit((const void *)build_slots_kernel, kMaxRequests * 16, done),
                       "build_slots: shared memory limit");
    const int64_t quads = (T + 3) / 4, work = quads > B ? quads : B;     // threads that have something to do
    // a CTA for 4096 rows or 32 requests (whose blocks may come back), whichever asks for more
    const int64_t most = in_place ? 8 : num_sms(), want = quads / 1024 + 1 > B / 32 ? quads / 1024 + 1 : B / 32;
    const int ctas = (int)(want < 1 ? 1 : (want < most ? want : most));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(work <= 128 ? 128 : (work <= 512 ? 512 : 1024));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream_of(stream);
    cudaLaunchAttribute at[2] = {pdl_attribute(), {}};
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = in_place ? ctas : 1;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = in_place ? 2 : 1;
    CSA2_CUDA_CALL(cudaLaunchKernelEx(&cfg, build_slots_kernel, args), "build_slots_kernel launch");
    CSA2_LAUNCH_CHECK("build_slots_kernel");
    return CSA2_OK;
}
