// evict.cu -- tv_evict_cache: keep each KV head's cache to a budget by the
// accumulated attention weights.
//
// Kept are the first `sink` tokens, the last `recent` ones and, of those
// between, the budget - sink - recent with the largest sums (equal sums: the
// lower position; a NaN ranks below every number).  The kept tokens keep their
// order: token kept[r] moves to position r.
//
// evict_select_kernel: one cluster per (sequence, KV head).  Each CTA reads its
// slice of the sums once and keeps them as order-preserving keys in shared memory;
// a radix selection (digits of 11, 11 and 10 bits, the CTAs' counts added up
// through distributed shared memory) finds the smallest kept key and how many
// of its equals are kept; then each warp writes the positions of its part in
// order, starting from the counts of the parts before it.
//
// evict_move_kernel: rows move from kept[r] to r.  In place a destination can
// be another row's source, but never a later one's: src(r) >= r, and src rises
// with r, so for r < r' the destination r <= r' - 1 < src(r').  One cluster per
// (sequence, KV head) takes the rows in ascending chunks; all of a chunk is
// read before any of it is written (a cluster barrier between), which with the
// inequality above is all that is needed.  From the chunk on whose first source
// lies past the last destination, nothing that is still to be read can be
// written any more, and the barriers end.  Copies into other blocks need no
// order and no barrier.
//
// Bound: the selection by its chain of some twenty dependent steps (about 7 us at
// 4,096 sums, 20 us at 131,072), the move by HBM: 8 x 8,190 tokens to 4,001,
// copied (267 MB), 58 us together, the move at 5.6 TB/s; 32 sequences of 512 to
// 32,768 to 4,096 in place (1.05 GB), 214 us.
#include <cooperative_groups.h>

#include "kernels.h"
#include "tv_common.cuh"

namespace cg = cooperative_groups;

namespace tv {
namespace {

constexpr int SE_THREADS = 512;
constexpr int SE_WARPS = SE_THREADS / 32;
constexpr int SE_MAX_CLUSTER = 16;
constexpr int SE_MAX_SLICE = 49152;  // sums in one CTA's shared memory (192 KB)
constexpr int BINS = 2048;
constexpr int SE_UN = 4;             // 16-byte loads of sums that a thread has in flight
constexpr int SE_STEP = 128;         // slices are multiples of this many sums

// Order-preserving key of a sum: larger sums, larger keys; NaN 0; -0 as +0.
__device__ __forceinline__ uint32_t sum_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.0f);  // -0 + 0 = +0
    return w != w ? 0u : u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
}
__device__ __forceinline__ float key_sum(uint32_t key) {
    return __uint_as_float(key == 0 ? 0x7fc00000u : key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// A predicated store (branches would keep the ones after it waiting).
__device__ __forceinline__ void store_if(bool yes, void* p, int32_t x) {
    asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %0, 0;\n @p st.global.s32 [%1], %2;\n}" ::"r"((int)yes), "l"(p),
                 "r"(x)
                 : "memory");
}

struct SelectShared {
    uint32_t own[BINS];         // this CTA's counts of the current digit
    uint32_t total[3][BINS];    // the cluster's; CTA c keeps those of bins c * BINS / C and on
    uint32_t scan[SE_WARPS];
    uint2 warp_cnt[SE_WARPS];   // kept for certain, equal to the threshold
    uint2 cta_cnt;              // the CTA's sums of those, read by its peers
    uint32_t digit, above, whole;  // the threshold's digit, the keys above it, whether all keys that have it are kept
    int bad;
};

__global__ void __launch_bounds__(SE_THREADS) evict_select_kernel(const __grid_constant__ EvictArgs a, int vec) {
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ __align__(16) SelectShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int bh = blockIdx.x / C, b = bh / a.Hkv, h = bh - b * a.Hkv;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t L = a.lens[b];
    if (tid == 0) s.bad = 0;
    for (int i = tid; i < BINS / 4; i += SE_THREADS) reinterpret_cast<uint4*>(s.own)[i] = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < 3 * BINS / 4; i += SE_THREADS)
        reinterpret_cast<uint4*>(&s.total[0][0])[i] = make_uint4(0, 0, 0, 0);
    int32_t* kept = a.kept + (size_t)bh * a.budget;
    const bool lead = h == 0 && rank == 0 && tid == 0;
    if (L < 0 || L > a.max_len) {  // the same in every CTA of the cluster
        if (lead) {
            a.new_lens[b] = L;
            report(a.status, TV_ERR_INVALID_ARG);
        }
        for (int r = rank * SE_THREADS + tid; r < a.budget; r += C * SE_THREADS) kept[r] = -1;
        return;
    }
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // the totals are cleared
    const int n = L < a.budget ? L : a.budget;
    const bool cut = L > a.budget;
    const int want = cut ? a.budget - a.sink - a.recent : 0;
    // candidates: lo <= t < lo + span, as one unsigned comparison
    const uint32_t lo = cut ? a.sink : 0, span = cut ? L - a.recent - a.sink : 0;
    // block ids of the span that is read and of the one that is written
    {
        const int32_t* bt = a.c.table + (size_t)b * a.c.max_blocks;
        const int32_t* dt = a.dst_table ? a.dst_table + (size_t)b * a.c.max_blocks : nullptr;
        const int nb = (int)(((int64_t)L + a.c.block_size - 1) / a.c.block_size);
        const int nd = dt ? (int)(((int64_t)n + a.c.block_size - 1) / a.c.block_size) : 0;
        int bad = 0;
        for (int i = rank * SE_THREADS + tid; i < nb; i += C * SE_THREADS)
            bad |= bt[i] < 0 || bt[i] >= a.c.num_blocks;
        for (int i = rank * SE_THREADS + tid; i < nd; i += C * SE_THREADS)
            bad |= dt[i] < 0 || dt[i] >= a.c.num_blocks;
        if (bad) s.bad = 1;
    }
    // this CTA's slice of the sums
    const int slice = ((L + C - 1) / C + SE_STEP - 1) / SE_STEP * SE_STEP;
    const int t0 = min(L, rank * slice), t1 = min(L, t0 + slice), len = t1 - t0;
    const float* w = a.weights + (size_t)bh * a.weight_stride + t0;
#pragma unroll 1
    for (int y0 = tid * 4; y0 < len; y0 += SE_UN * 4 * SE_THREADS) {
        float4 x[SE_UN];
#pragma unroll
        for (int i = 0; i < SE_UN; ++i) {
            const int y = y0 + i * 4 * SE_THREADS;
            if (vec && y + 4 <= len) {
                x[i] = *reinterpret_cast<const float4*>(w + y);
            } else {
                x[i].x = y < len ? w[y] : 0.f;
                x[i].y = y + 1 < len ? w[y + 1] : 0.f;
                x[i].z = y + 2 < len ? w[y + 2] : 0.f;
                x[i].w = y + 3 < len ? w[y + 3] : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < SE_UN; ++i) {
            const int y = y0 + i * 4 * SE_THREADS;
            if (y >= len) break;
            const uint4 k = make_uint4(sum_key(x[i].x), sum_key(x[i].y), sum_key(x[i].z), sum_key(x[i].w));
            *reinterpret_cast<uint4*>(s_key + y) = k;
            const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (want && (uint32_t)(t0 + y + e) - lo < span && y + e < len) atomicAdd(&s.own[ks[e] >> 21], 1u);
        }
    }
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    // the smallest kept key, and how many of its equals are kept; none when only sink and recent are
    uint32_t threshold = want ? 0u : 0xffffffffu, left = (uint32_t)want;
    if (want) {
        constexpr int PER = 4;
        static_assert(PER * SE_THREADS == BINS, "four bins per thread");
        const int bin0 = BINS - PER - PER * tid;  // bins from the top down: this thread's are bin0 .. bin0 + 3
        const int owner = bin0 / (BINS / C);
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            if (pass) {
                const int shift = pass == 1 ? 10 : 0, done = pass == 1 ? 21 : 10;
                const uint32_t mask = pass == 1 ? 2047u : 1023u;
#pragma unroll 1
                for (int y = tid * 4; y < len; y += 4 * SE_THREADS) {
                    const uint4 k = *reinterpret_cast<const uint4*>(s_key + y);
                    const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((ks[e] ^ threshold) >> done == 0 && (uint32_t)(t0 + y + e) - lo < span && y + e < len)
                            atomicAdd(&s.own[(ks[e] >> shift) & mask], 1u);
                }
                __syncthreads();
            }
            uint4 cnt = *reinterpret_cast<const uint4*>(&s.own[bin0]);
            if (C > 1) {
                // bins that hold any go to the CTA that keeps their totals; then everybody reads all totals
                if (cnt.x | cnt.y | cnt.z | cnt.w) {
                    uint32_t* to = cluster.map_shared_rank(&s.total[pass][bin0], owner);
                    if (cnt.x) atomicAdd(to, cnt.x);
                    if (cnt.y) atomicAdd(to + 1, cnt.y);
                    if (cnt.z) atomicAdd(to + 2, cnt.z);
                    if (cnt.w) atomicAdd(to + 3, cnt.w);
                }
                cluster.sync();
                cnt = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&s.total[pass][bin0], owner));
            }
            *reinterpret_cast<uint4*>(&s.own[bin0]) = make_uint4(0, 0, 0, 0);
            const uint32_t sum = cnt.x + cnt.y + cnt.z + cnt.w;
            uint32_t inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) s.scan[warp] = inc;
            __syncthreads();
            uint32_t before = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? s.scan[lane] : 0u);
            if (before < left && left <= before + sum) {
                const uint32_t c[4] = {cnt.w, cnt.z, cnt.y, cnt.x};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (before < left && left <= before + c[e]) {
                        s.digit = bin0 + 3 - e;
                        s.above = before;
                        s.whole = left == before + c[e];
                    }
                    before += c[e];
                }
            }
            __syncthreads();
            threshold |= s.digit << (pass == 0 ? 21 : pass == 1 ? 10 : 0);
            left -= s.above;
            if (s.whole) {  // every key that begins like this is kept, whatever its other digits: the usual end
                --threshold;  // not 0: there are more candidates than are kept
                left = 0;
                break;
            }
        }
    }
    // kept for certain: not a candidate, or above the threshold
    auto sure = [&](int y, uint32_t key) { return (uint32_t)(t0 + y) - lo >= span || key > threshold; };
    const int per = ((len + SE_WARPS - 1) / SE_WARPS + 31) / 32 * 32;
    const int w0 = min(len, warp * per), w1 = min(len, w0 + per);  // this warp's part of the slice
    uint32_t nk = 0, ne = 0;
#pragma unroll 4
    for (int y = w0 + lane; y < w1; y += 32) {
        const uint32_t key = s_key[y];
        const bool k = sure(y, key);
        nk += k;
        ne += !k && key == threshold;
    }
    nk = __reduce_add_sync(0xffffffffu, nk);
    ne = __reduce_add_sync(0xffffffffu, ne);
    if (lane == 0) s.warp_cnt[warp] = make_uint2(nk, ne);
    __syncthreads();
    // before this warp: kept for certain, equals
    const uint2 wc = lane < SE_WARPS ? s.warp_cnt[lane] : make_uint2(0, 0);
    uint32_t bk = __reduce_add_sync(0xffffffffu, lane < warp ? wc.x : 0u);
    uint32_t be = __reduce_add_sync(0xffffffffu, lane < warp ? wc.y : 0u);
    int bad = s.bad;
    if (C > 1) {
        if (warp == 0) {
            const uint32_t k = __reduce_add_sync(0xffffffffu, wc.x), e = __reduce_add_sync(0xffffffffu, wc.y);
            if (lane == 0) s.cta_cnt = make_uint2(k, e);
        }
        cluster.sync();  // every slice is in shared memory: the sums may be overwritten
        uint2 pc = make_uint2(0, 0);
        int pb = 0;
        if (lane < C) {
            pc = *cluster.map_shared_rank(&s.cta_cnt, lane);
            pb = *cluster.map_shared_rank(&s.bad, lane);
        }
        bk += __reduce_add_sync(0xffffffffu, lane < rank ? pc.x : 0u);
        be += __reduce_add_sync(0xffffffffu, lane < rank ? pc.y : 0u);
        bad = __any_sync(0xffffffffu, pb);
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    if (bad) {
        if (lead) {
            a.new_lens[b] = L;
            report(a.status, TV_ERR_BLOCK_TABLE);
        }
        for (int r = rank * SE_THREADS + tid; r < a.budget; r += C * SE_THREADS) kept[r] = -1;
    } else {
        float* wo = a.weights_out ? a.weights_out + (size_t)bh * a.weight_stride : nullptr;
        const uint32_t below = (1u << lane) - 1;
        // Four groups of 32 positions at once, one position per lane: the votes' latencies overlap.
#pragma unroll 1
        for (int y0 = w0; y0 < w1; y0 += 128) {
            uint32_t key[4], r[4], equal = 0;
            bool take[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int y = y0 + 32 * e + lane;
                key[e] = y < w1 ? s_key[y] : 0;
                take[e] = y < w1 && sure(y, key[e]);
                equal |= (uint32_t)(y < w1 && !take[e] && key[e] == threshold) << e;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t kb = __ballot_sync(0xffffffffu, take[e]);
                r[e] = bk + __popc(kb & below);
                bk += __popc(kb);
            }
            if (left) {  // equals of the threshold: the first `left` of them
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool eq = equal >> e & 1;
                    const uint32_t eb = __ballot_sync(0xffffffffu, eq), mine = be + __popc(eb & below);
                    take[e] |= eq && mine < left;
                    r[e] += min(mine, left);
                    be += __popc(eb);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                store_if(take[e], kept + r[e], t0 + y0 + 32 * e + lane);
                store_if(take[e] && wo, wo + r[e], (int32_t)__float_as_uint(key_sum(key[e])));
            }
        }
        for (int r = n + rank * SE_THREADS + tid; r < a.budget; r += C * SE_THREADS) kept[r] = -1;
        if (wo) {
            const int z0 = max(t0, n), zv = vec ? min(t1, (z0 + 3) / 4 * 4) : t1;  // vec: then rows of sums are 16-byte aligned
            if (!vec)
                for (int t = z0 + tid; t < t1; t += SE_THREADS) wo[t] = 0.f;
            else if (tid < 4 && z0 + tid < zv) wo[z0 + tid] = 0.f;
            for (int t = zv + tid * 4; t < t1; t += 4 * SE_THREADS) {
                if (t + 4 <= t1) *reinterpret_cast<float4*>(wo + t) = make_float4(0.f, 0.f, 0.f, 0.f);
                else
                    for (int e = t; e < t1; ++e) wo[e] = 0.f;
            }
        }
        if (lead) a.new_lens[b] = n;
    }
    __syncwarp();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no peer reads this CTA's counts any more
}

constexpr int MV_WARPS = 8;
constexpr int MV_THREADS = MV_WARPS * 32;
constexpr int MV_STAGE = 4096;  // bytes of a warp's step
constexpr int MV_STAGES = 2;

__device__ __forceinline__ void mv_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}

// Work of `ctas` CTAs (a cluster in place): the K rows or the V rows of one (sequence, KV head).
template <bool IN_PLACE>
__global__ void __launch_bounds__(MV_THREADS) evict_move_kernel(const __grid_constant__ EvictArgs a, int ctas) {
    extern __shared__ __align__(16) uint4 mv_ring[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int unit = blockIdx.x / ctas, part = blockIdx.x - unit * ctas, bh = unit / 2, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int32_t L = a.lens[b];
    const int n = L < 0 || L > a.max_len ? 0 : min(L, a.budget);
    const int32_t* kept = a.kept + (size_t)bh * a.budget;
    const int32_t* bt = a.c.table + (size_t)b * a.c.max_blocks;
    const int32_t* dt = IN_PLACE ? bt : a.dst_table + (size_t)b * a.c.max_blocks;
    const int cpr = a.row_bytes / 16;
    const int rows = min(32, MV_STAGE / a.row_bytes);  // rows of a warp's step, one lane's offsets each
    char* base = static_cast<char*>(unit & 1 ? a.v : a.k) + (int64_t)h * a.c.head_stride;
    uint4* ring = mv_ring + warp * (MV_STAGES * MV_STAGE / 16);
    const int chunk = rows * MV_WARPS * ctas, first = (part * MV_WARPS + warp) * rows;
    const int pieces = rows * cpr, drow = 32 / cpr, dpiece = 32 - drow * cpr;
    const int row0 = lane / cpr, piece0 = lane - row0 * cpr;
    const int steps = (n + chunk - 1) / chunk;
    // lane's row of step s: where it goes to (-1: there is none), and where it comes from (-1: nothing to move)
    auto target = [&](int s) -> int64_t {
        const int r = s * chunk + first + lane;
        if (lane >= rows || r >= n) return -1;
        const int blk = r / a.c.block_size, id = dt[blk];
        if (id < 0 || id >= a.c.num_blocks) return -1;  // the selection reports it
        return (int64_t)id * a.c.block_stride + (int64_t)(r - blk * a.c.block_size) * a.c.token_stride;
    };
    auto source = [&](int s) -> int64_t {
        const int r = s * chunk + first + lane;
        if (lane >= rows || r >= n) return -1;
        const int t = kept[r];
        if (t < 0 || t >= L || (IN_PLACE && t == r)) return -1;  // a flagged sequence, or in place already
        const int blk = t / a.c.block_size;
        return (int64_t)bt[blk] * a.c.block_stride + (int64_t)(t - blk * a.c.block_size) * a.c.token_stride;
    };
    auto load = [&](int stage, int64_t src) {
        int row = row0, piece = piece0;
        for (int x = lane; x - lane < pieces; x += 32) {
            const int64_t o = __shfl_sync(0xffffffffu, src, row & 31);
            if (x < pieces && o >= 0) mv_async16(ring + stage * (MV_STAGE / 16) + x, base + o + piece * 16);
            row += drow;
            piece += dpiece;
            if (piece >= cpr) {
                piece -= cpr;
                ++row;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the targets do not depend on the selection
    int64_t dst = target(0), dst_next = target(1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n == 0 || (IN_PLACE && n == L)) return;  // nothing moves: the same for the whole cluster
    int64_t src = source(0), src_next = source(1);
    // where the first row of a step (of all CTAs) comes from: the others come from behind it
    auto head_of = [&](int s) { return (int64_t)s * chunk < n ? kept[s * chunk] : n; };
    int head = IN_PLACE ? kept[0] : n, head_next = IN_PLACE ? head_of(1) : n;
    load(0, src);
    for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps) load((s + 1) % MV_STAGES, src_next);
        else asm volatile("cp.async.commit_group;" ::: "memory");
        const int64_t src_now = src, dst_now = dst;
        src = src_next;
        dst = dst_next;
        dst_next = target(s + 2);
        src_next = source(s + 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        if (IN_PLACE && head < n) {  // all of this step has been read; no barrier once the sources lie past every target
            if (ctas > 1) cg::this_cluster().sync();
            else __syncthreads();
            head = head_next;
            head_next = head_of(s + 2);
        }
        int row = row0, piece = piece0;
        const uint4* st = ring + (s % MV_STAGES) * (MV_STAGE / 16);
        for (int x = lane; x - lane < pieces; x += 32) {
            const int64_t o = __shfl_sync(0xffffffffu, src_now < 0 ? -1 : dst_now, row & 31);
            if (x < pieces && o >= 0) *reinterpret_cast<uint4*>(base + o + piece * 16) = st[x];
            row += drow;
            piece += dpiece;
            if (piece >= cpr) {
                piece -= cpr;
                ++row;
            }
        }
        __syncwarp();
    }
}

cudaError_t launch(const void* kern, unsigned grid, int cluster, int threads, size_t smem, bool dependent,
                   cudaStream_t st, void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

}  // namespace

int evict_max_len() { return SE_MAX_CLUSTER * SE_MAX_SLICE; }

cudaError_t launch_evict(const EvictArgs& a, int sms, cudaStream_t st) {
    const int heads = a.B * a.Hkv;
    // Slices of 2,048 to 4,096 sums (four to eight for each thread), as long as the GPU holds twice
    // the CTAs at four per SM.  At 128K sums and 8 heads clusters of 4, 8 and 16 took (with the move) 63, 50
    // and 49 us; above 8, which not every part of the GPU can place, only for what would not fit.
    int C = 1;
    while (C < 8 && (int64_t)C * 4096 < a.max_len && (int64_t)heads * C * 2 <= 4 * sms) C *= 2;
    while ((int64_t)C * SE_MAX_SLICE < a.max_len) C *= 2;
    const size_t smem = sizeof(uint32_t) * ((((size_t)a.max_len + C - 1) / C + SE_STEP - 1) / SE_STEP * SE_STEP);
    static SmemLimit limit;  // the largest slice's, for every call
    cudaError_t e = limit.allow((const void*)evict_select_kernel, (int)sizeof(float) * SE_MAX_SLICE);
    if (e == cudaSuccess && C > 8)
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int vec = a.weight_stride % 4 == 0 &&
              !((reinterpret_cast<uintptr_t>(a.weights) | reinterpret_cast<uintptr_t>(a.weights_out)) & 15);
    void* args[] = {const_cast<EvictArgs*>(&a), &vec};
    e = launch((const void*)evict_select_kernel, (unsigned)(heads * C), C, SE_THREADS, smem, false, st, args);
    if (e != cudaSuccess) return e;
    const int rows = (MV_STAGE / a.row_bytes < 32 ? MV_STAGE / a.row_bytes : 32) * MV_WARPS;  // of a CTA's step
    int ctas = 1;
    const int most = a.budget < a.max_len ? a.budget : a.max_len;  // rows of a head
    const int ring = MV_WARPS * MV_STAGES * MV_STAGE;
    void* margs[] = {const_cast<EvictArgs*>(&a), &ctas};
    // Steps of 4 KB in 8 warps.  Selection and move together, four cases (4K in place, 8 x 8K
    // copied, 128K copied, 32 mixed in place): 13.0, 57.7, 46.6 and 214 us; 4 KB in 4 warps 15.5,
    // 57.1, 46.4 and 225; 2 KB in 8 warps 14.9, 61, 46.5 and 229; 8 KB in 4 warps 13.5, 60, 48.3 and 225.
    // Copies: two steps per CTA (one 64 us at 8 x 8K, three 60).  In place: a cluster of up to 8,
    // while the GPU has no 8 CTAs per SM (4: 227 us on the mixed case, 16: 232).
    if (a.dst_table) {
        ctas = (most + 2 * rows - 1) / (2 * rows);
        static SmemLimit copy_limit;
        e = copy_limit.allow((const void*)evict_move_kernel<false>, ring);
        if (e != cudaSuccess) return e;
        return launch((const void*)evict_move_kernel<false>, (unsigned)(2 * heads * ctas), 1, MV_THREADS, ring, true, st,
                      margs);
    }
    while (ctas < 8 && ctas * rows < most && (int64_t)2 * heads * ctas < 8LL * sms) ctas *= 2;
    static SmemLimit place_limit;
    e = place_limit.allow((const void*)evict_move_kernel<true>, ring);
    if (e != cudaSuccess) return e;
    return launch((const void*)evict_move_kernel<true>, (unsigned)(2 * heads * ctas), ctas, MV_THREADS, ring, true, st,
                  margs);
}

}  // namespace tv
