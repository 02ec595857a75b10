// evict.cu -- tv_evict_cache: keep each KV head's cache to a budget by the
// accumulated attention weights.
//
// Kept are the first `sink` tokens, the last `recent` ones and, of those
// between, the budget - sink - recent with the largest sums (equal sums: the
// lower position; a NaN ranks below every number).  The kept tokens keep their
// order: token kept[r] moves to position r.
//
// evict_select_kernel: one cluster per (sequence, KV head).  Each CTA reads its
// slice of the sums into shared memory once; a radix selection (digits of 11,
// 11 and 10 bits of the order-preserving key, histograms joined through
// distributed shared memory) finds the smallest kept key and how many of its
// equals are kept; then each warp writes the positions of its part in order
// (ballots), starting from the counts of the parts before it.
//
// evict_move_kernel: rows move from kept[r] to r.  In place a destination can
// be another row's source, but never a later one's: src(r) >= r, and src rises
// with r, so for r < r' the destination r <= r' - 1 < src(r').  One cluster per
// (sequence, KV head) takes the rows in ascending chunks; all of a chunk is
// read before any of it is written (a cluster barrier between), which with the
// inequality above is all that is needed.  Copies into other blocks need no
// order and no barrier.
#include <cooperative_groups.h>

#include "kernels.h"
#include "tv_common.cuh"

namespace cg = cooperative_groups;

namespace tv {
namespace {

constexpr int SE_THREADS = 512;
constexpr int SE_WARPS = SE_THREADS / 32;
constexpr int SE_MAX_CLUSTER = 16;
constexpr int SE_MAX_SLICE = 51200;  // sums in one CTA's shared memory (200 KB)
constexpr int BINS = 2048;

// Order-preserving key of a sum: larger sums, larger keys; NaN 0; -0 as +0.
__device__ __forceinline__ uint32_t sum_key(float w) {
    if (w != w) return 0;
    const uint32_t u = __float_as_uint(w + 0.0f);  // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelectShared {
    uint32_t hist[3][BINS];
    uint32_t scan[SE_WARPS + 1];
    uint32_t wgt[SE_WARPS], weq[SE_WARPS];   // kept for certain / equal to the threshold, per warp
    uint32_t cta_keep, cta_eq;               // the CTA's counts, read by its peers
    uint32_t digit, above;
    int bad;
};

__global__ void __launch_bounds__(SE_THREADS) evict_select_kernel(const __grid_constant__ EvictArgs a) {
    extern __shared__ float s_w[];
    __shared__ SelectShared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int bh = blockIdx.x / C, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int32_t L = a.lens[b];
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
    const int n = L < a.budget ? L : a.budget;
    if (tid == 0) s.bad = 0;
    for (int i = tid; i < 3 * BINS; i += SE_THREADS) (&s.hist[0][0])[i] = 0;
    __syncthreads();
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
    const int slice = (L + C - 1) / C;
    const int t0 = min(L, rank * slice), t1 = min(L, t0 + slice);
    const float* w = a.weights + (size_t)bh * a.weight_stride;
    const int lo = min(a.sink, L), hi = max(lo, L - a.recent);  // candidates [lo, hi)
    const bool cut = L > a.budget;
    const int want = cut ? a.budget - a.sink - a.recent : 0;
    for (int t = t0 + tid; t < t1; t += SE_THREADS) {
        const float x = w[t];
        s_w[t - t0] = x;
        if (want && t >= lo && t < hi) atomicAdd(&s.hist[0][sum_key(x) >> 21], 1u);
    }
    cluster.sync();
    int bad = 0;
    for (int c = 0; c < C; ++c) bad |= *cluster.map_shared_rank(&s.bad, c);
    uint32_t prefix = 0, left = (uint32_t)want;  // key bits found so far; how many are still to be taken
    if (want && !bad) {
        constexpr int PER = BINS / SE_THREADS;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            if (pass) {
                const int shift = pass == 1 ? 10 : 0, keep_shift = pass == 1 ? 21 : 10;
                const uint32_t mask = pass == 1 ? 2047u : 1023u;
                for (int t = max(t0, lo) + tid; t < min(t1, hi); t += SE_THREADS) {
                    const uint32_t key = sum_key(s_w[t - t0]);
                    if ((key ^ prefix) >> keep_shift == 0) atomicAdd(&s.hist[pass][(key >> shift) & mask], 1u);
                }
                cluster.sync();
            }
            // bins from the top down: thread i holds bins BINS - 1 - PER i and below
            uint32_t cnt[PER], sum = 0;
#pragma unroll
            for (int e = 0; e < PER; ++e) cnt[e] = 0;
            for (int c = 0; c < C; ++c) {
                const uint32_t* peer = cluster.map_shared_rank(&s.hist[pass][0], c);
#pragma unroll
                for (int e = 0; e < PER; ++e) cnt[e] += peer[BINS - 1 - (PER * tid + e)];
            }
#pragma unroll
            for (int e = 0; e < PER; ++e) sum += cnt[e];
            uint32_t inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) s.scan[warp] = inc;
            __syncthreads();
            uint32_t before = inc - sum;
            for (int x = 0; x < warp; ++x) before += s.scan[x];
            if (before < left && left <= before + sum) {
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    if (before < left && left <= before + cnt[e]) {
                        s.digit = BINS - 1 - (PER * tid + e);
                        s.above = before;
                    }
                    before += cnt[e];
                }
            }
            __syncthreads();
            prefix |= s.digit << (pass == 0 ? 21 : pass == 1 ? 10 : 0);
            left -= s.above;
            __syncthreads();
        }
    }
    // prefix is now the smallest kept key, left how many of its equals are kept
    const bool select = cut && !bad;
    auto sure = [&](int t, uint32_t key) {
        return !cut || t < lo || t >= hi || (want && key > prefix);
    };
    const int per = ((t1 - t0 + SE_WARPS - 1) / SE_WARPS + 31) / 32 * 32;
    const int w0 = min(t1, t0 + warp * per), w1 = min(t1, w0 + per);
    uint32_t nk = 0, ne = 0;
    for (int t = w0 + lane; t - lane < w1; t += 32) {
        const bool in = t < w1;
        const uint32_t key = in ? sum_key(s_w[t - t0]) : 0;
        const bool k = in && sure(t, key);
        const bool e = in && !k && select && want && key == prefix;
        nk += __popc(__ballot_sync(0xffffffffu, k));
        ne += __popc(__ballot_sync(0xffffffffu, e));
    }
    if (lane == 0) {
        s.wgt[warp] = nk;
        s.weq[warp] = ne;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t k = 0, e = 0;
        for (int x = 0; x < SE_WARPS; ++x) {
            k += s.wgt[x];
            e += s.weq[x];
        }
        s.cta_keep = k;
        s.cta_eq = e;
    }
    cluster.sync();  // every slice is in shared memory: the sums may be overwritten
    uint32_t bk = 0, be = 0;  // before this warp: kept for certain, equals
    for (int c = 0; c < rank; ++c) {
        bk += *cluster.map_shared_rank(&s.cta_keep, c);
        be += *cluster.map_shared_rank(&s.cta_eq, c);
    }
    cluster.sync();  // no CTA leaves while a peer reads its counts
    if (bad) {
        if (lead) {
            a.new_lens[b] = L;
            report(a.status, TV_ERR_BLOCK_TABLE);
        }
        for (int r = rank * SE_THREADS + tid; r < a.budget; r += C * SE_THREADS) kept[r] = -1;
        return;
    }
    for (int x = 0; x < warp; ++x) {
        bk += s.wgt[x];
        be += s.weq[x];
    }
    float* wo = a.weights_out ? a.weights_out + (size_t)bh * a.weight_stride : nullptr;
    for (int t = w0 + lane; t - lane < w1; t += 32) {
        const bool in = t < w1;
        const float x = in ? s_w[t - t0] : 0.f;
        const uint32_t key = in ? sum_key(x) : 0;
        const bool k = in && sure(t, key);
        const bool e = in && !k && select && want && key == prefix;
        const uint32_t kb = __ballot_sync(0xffffffffu, k), eb = __ballot_sync(0xffffffffu, e);
        const uint32_t below = (1u << lane) - 1;
        const uint32_t my_eq = be + __popc(eb & below);  // equals before this one
        if (k || (e && my_eq < left)) {
            const uint32_t r = bk + __popc(kb & below) + min(my_eq, left);
            kept[r] = t;
            if (wo) wo[r] = x;
        }
        bk += __popc(kb);
        be += __popc(eb);
    }
    for (int r = n + rank * SE_THREADS + tid; r < a.budget; r += C * SE_THREADS) kept[r] = -1;
    if (wo)
        for (int t = max(t0, n) + tid; t < t1; t += SE_THREADS) wo[t] = 0.f;
    if (lead) a.new_lens[b] = n;
}

constexpr int MV_THREADS = 256;
constexpr int MV_UN = 8;                      // 16-byte pieces in flight per thread
constexpr int MV_PIECES = MV_THREADS * MV_UN;  // pieces per CTA and chunk

__global__ void __launch_bounds__(MV_THREADS) evict_move_kernel(const __grid_constant__ EvictArgs a, int rows_per_cta,
                                                                int ctas) {
    const bool in_place = a.dst_table == nullptr;
    const int tid = threadIdx.x;
    // in place: one cluster of `ctas` walks the head's rows; else `ctas` independent CTAs share them
    const int bh = blockIdx.x / ctas, part = blockIdx.x - bh * ctas, b = bh / a.Hkv, h = bh - b * a.Hkv;
    const int32_t L = a.lens[b];
    if (L < 0 || L > a.max_len) return;
    const int n = L < a.budget ? L : a.budget;
    if (in_place && n == L) return;  // nothing moves
    const int32_t* kept = a.kept + (size_t)bh * a.budget;
    if (n == 0 || kept[0] < 0) return;  // flagged by the selection
    const int32_t* bt = a.c.table + (size_t)b * a.c.max_blocks;
    const int32_t* dt = in_place ? bt : a.dst_table + (size_t)b * a.c.max_blocks;
    const int cpr = a.row_bytes / 16;
    const int64_t head = (int64_t)h * a.c.head_stride;
    auto row_off = [&](const int32_t* tab, int t) {
        const int blk = t / a.c.block_size;
        return (int64_t)tab[blk] * a.c.block_stride + (int64_t)(t - blk * a.c.block_size) * a.c.token_stride + head;
    };
    const int chunk = rows_per_cta * ctas;
    for (int r0 = 0; r0 < n; r0 += chunk) {
        const int first = r0 + part * rows_per_cta;
        uint4 buf[MV_UN];
        int64_t to[MV_UN];
#pragma unroll
        for (int i = 0; i < MV_UN; ++i) {
            const int x = i * MV_THREADS + tid;
            const int row = x / (2 * cpr), y = x - row * 2 * cpr;  // y: piece of the K row, then of the V row
            const int r = first + row;
            to[i] = -1;
            if (row < rows_per_cta && r < n) {
                const int src = kept[r];
                if (!in_place || src != r) {
                    const bool isv = y >= cpr;
                    const int64_t piece = (int64_t)(isv ? y - cpr : y) * 16;
                    buf[i] = *reinterpret_cast<const uint4*>(static_cast<const char*>(isv ? a.v : a.k) +
                                                             row_off(bt, src) + piece);
                    to[i] = row_off(dt, r) + piece;
                }
            }
        }
        if (in_place) {
            if (ctas > 1) cg::this_cluster().sync();
            else __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < MV_UN; ++i) {
            const int x = i * MV_THREADS + tid;
            const int row = x / (2 * cpr), y = x - row * 2 * cpr;
            if (to[i] >= 0)
                *reinterpret_cast<uint4*>(static_cast<char*>(y >= cpr ? a.v : a.k) + to[i]) = buf[i];
        }
    }
}

cudaError_t launch_cluster(const void* kern, unsigned grid, int cluster, int threads, size_t smem, cudaStream_t st,
                           void** args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

}  // namespace

int evict_max_len() { return SE_MAX_CLUSTER * SE_MAX_SLICE; }

cudaError_t launch_evict(const EvictArgs& a, int sms, cudaStream_t st) {
    const int heads = a.B * a.Hkv;
    int C = 1;
    while (C < 8 && (int64_t)C * 4096 < a.max_len && (int64_t)heads * C < 2 * sms) C *= 2;
    while ((int64_t)C * SE_MAX_SLICE < a.max_len) C *= 2;
    const size_t smem = sizeof(float) * (((size_t)a.max_len + C - 1) / C);
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && C > 8)
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    void* args[] = {const_cast<EvictArgs*>(&a)};
    e = launch_cluster((const void*)evict_select_kernel, (unsigned)(heads * C), C, SE_THREADS, smem, st, args);
    if (e != cudaSuccess) return e;
    const int cpr = a.row_bytes / 16;
    int rows = MV_PIECES / (2 * cpr);
    int ctas = 1;
    if (a.dst_table) {
        const int64_t all = (a.budget + rows - 1) / rows;
        ctas = (int)all;
        while (ctas > 1 && (int64_t)heads * ctas > 16LL * sms) ctas = (ctas + 1) / 2;
    } else {
        while (ctas < 8 && ctas * rows < a.budget && (int64_t)heads * ctas < 4LL * sms) ctas *= 2;
    }
    void* margs[] = {const_cast<EvictArgs*>(&a), &rows, &ctas};
    return launch_cluster((const void*)evict_move_kernel, (unsigned)(heads * ctas), a.dst_table ? 1 : ctas, MV_THREADS, 0,
                          st, margs);
}

}  // namespace tv
