// decode.cu -- tv_decode_attention: one new token of every sequence attends to
// its paged cache.
//
//   s_t = scale q . k_t,   out = sum_t exp(s_t - lse) v_t,   lse = log sum_t exp(s_t)
//
// and, when asked for, weights[b][h][t] += sum over the KV head's query heads
// of exp(s_t - lse).
//
// Split.  The whole batch's work is one line of 16-token tiles, sequence by
// sequence and KV head by KV head; every CTA takes an equal stretch of it,
// whatever the sequences' lengths.  A stretch covers some heads whole (their
// result is final) and at most two in part: those leave their running maximum,
// sum and unnormalised output in the workspace, and a second kernel joins
// them in stretch order (so the result does not depend on timing).
//
// Inside a CTA the warps take tiles in turn.  Each warp keeps its own ring
// of tiles (cp.async, two or three deep) and its own running softmax, so there is no
// block barrier in the loop.
//
// bf16 and fp16 use warp-level matrix instructions (m16n8k16): S^T = K Q^T with
// the tokens as rows and up to 8 query heads as columns, then O^T += V^T P^T; the
// transposed 8x8 blocks of P come from movmatrix.  P goes into the product as a
// high and a low 16-bit part, which hold a weight to 2^-16 (bf16) or better: well
// below the rounding of the output (0.4 % of a ragged batch's bf16 outputs round
// differently from the exact ones, 0.14 % with fp32 weights).  The second product
// costs nothing, as the bytes of K and V bound this kernel, not the matrix units.
// The exponentials' reference
// is not the running maximum itself: it lies 2^7 below one and moves only when a
// score passes it by more than 2^15, so most tiles need no shuffles and no
// rescaling.  P stays below 2^15 (inside fp16, whose small values keep seven more
// bits than with a reference at the maximum) and the sums far inside fp32.  fp32
// runs on the CUDA cores (two lanes per token for the scores, lanes over the
// head's dimensions for the values).
//
// Bound: HBM.  32 sequences of 512 to 32,768 tokens (2.32 GB): 376 us, 94 % of the
// copy bandwidth; one of 131,072 with weights (545 MB): 112 us, of which the
// first kernel takes about 94 and the weights' pass the rest; one of 4,096
// (16.8 MB): 9.4 us, where launches and dependent loads count.  fp32 heads, 8 x 8,192
// tokens, 64/8 heads: 82, 119, 147 and 368 us at head_dim 64, 96, 128 and 256, that is 50,
// 52, 56 and 45 % of the copy bandwidth: the loop's instructions bound them (for each
// head and tile four dependent shuffles for the maximum, the queries read again from
// shared memory, a few spilled registers), at 3 to 8 warps per SM.  More query heads per
// KV head than one unit holds read K and V once per unit: fp32, 64/4 heads at head_dim 256,
// two units, 368 us, 22 %; bf16, 128/4 heads at 128, two units, 53 us, 39 %.
#include <cooperative_groups.h>

#include "kernels.h"
#include "tv_common.cuh"

namespace cg = cooperative_groups;

namespace tv {
namespace {

constexpr int TILE = 16;              // tokens per step of a warp
constexpr int MIN_TILES = 8;          // a CTA's shortest stretch
constexpr float LN2 = 0.6931471805599453f;
// 16-bit path: the exponentials' reference lies 2^7 below the largest score it was set by, and
// moves when a score passes it by more than 2^15.
constexpr float REF_BELOW = 7.f, REF_MOVES = 15.f;
constexpr float BAD_SUM = -1.f;       // sum of a piece whose block table is out of range

template <typename T, int D> struct Shape {
    // Rows are padded so that the eight rows of one ldmatrix (16-bit types), or the
    // four tokens times two halves of one 8-lane phase (fp32), fall into different banks.
    static constexpr int ROW = D * (int)sizeof(T) + (sizeof(T) == 2 ? 16 : 32);
    static constexpr int CH = D * (int)sizeof(T) / 16;  // 16-byte pieces of a row
    static constexpr int STAGE = 2 * TILE * ROW;        // a tile of K and of V
    static constexpr int STAGES = sizeof(T) == 2 ? 3 : 2;  // ring depth of a warp, in tiles
    static constexpr int RING = STAGES * STAGE;         // one warp's ring
    // Warps per CTA: 16-bit types four, for two CTAs per SM at head_dim 128; fp32 as many as fit.
    static constexpr int FIT = 210 * 1024 / RING;
    static constexpr int NW = sizeof(T) == 2 ? 4 : FIT < 8 ? FIT : 8;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// K and V pass through L2 once: first to leave, so that scores and partial results stay.
__device__ __forceinline__ uint64_t stream_policy() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
                 "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <typename T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
    static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    // two values as a pair of high parts and a pair of what those leave
    static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = *reinterpret_cast<const uint32_t*>(&l);
    }
};
template <> struct Mma<__half> {
    static __device__ __forceinline__ void run(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = *reinterpret_cast<const uint32_t*>(&l);
    }
};

// Tiles of sequence b (0 for a length out of range, which is reported elsewhere).
__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int b) {
    const int L = a.lens[b];
    return L < 0 || L > a.max_len ? 0 : (L + TILE - 1) / TILE;
}

// The CTA's stretch [pos, end) of the line and where it starts.
struct Start {
    int total;   // tiles of the whole line
    int b, cum;  // sequence that holds pos, and the tiles (per unit) before it
};

// Block-wide: thread i sums a run of sequences, the runs are scanned, and the
// thread whose run holds `pos` walks it.
template <int NW, typename F>
__device__ __forceinline__ void find_start(const DecodeArgs& a, int units, F pos_of, bool write_cum, Start* s_start,
                                           int* s_scan) {
    constexpr int DE_THREADS = NW * 32;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int run = (a.B + DE_THREADS - 1) / DE_THREADS;
    const int b0 = min(a.B, tid * run), b1 = min(a.B, b0 + run);
    int sum = 0;
    for (int b = b0; b < b1; ++b) sum += tiles_of(a, b);
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    int before = inc - sum, all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += s_scan[w];
        all += s_scan[w];
    }
    const int total = all * units;
    const int pos = pos_of(total);
    if (write_cum) {
        int c = before;
        for (int b = b0; b < b1; ++b) {
            a.cum[b] = c;
            c += tiles_of(a, b);
        }
        if (tid == 0) a.cum[a.B] = all;
    }
    if (tid == 0) s_start->total = total;
    if (pos < total && pos >= before * units && pos < (before + sum) * units) {
        int b = b0, c = before;
        for (;; ++b) {
            const int t = tiles_of(a, b);
            if (pos < (c + t) * units) break;
            c += t;
        }
        s_start->b = b;
        s_start->cum = c;
    }
    __syncthreads();
}

__device__ __forceinline__ int stretch(int total, int grid) {
    const int per = (total + grid - 1) / grid;
    return per < MIN_TILES ? MIN_TILES : per;
}

// CLUSTERS: a unit's tiles are shared by the CTAs of one cluster, which join their parts
// through each other's shared memory and add the weights themselves: one launch.
template <typename T, int D, int HT, bool CLUSTERS>
__global__ void __launch_bounds__(Shape<T, D>::NW * 32) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using S = Shape<T, D>;
    constexpr int NW = S::NW, DE_THREADS = NW * 32;
    constexpr bool MMA = sizeof(T) == 2;
    constexpr int NT = MMA ? HT / 8 : 1;
    constexpr int KS = D / 16;
    constexpr int DV = D / 32;  // values per lane on the fp32 path
    extern __shared__ __align__(16) unsigned char ring_all[];
    __shared__ Start s_start;
    __shared__ int s_scan[NW];
    __shared__ float s_m[NW][HT], s_l[NW][HT];
    __shared__ float2 s_ml[CLUSTERS ? HT : 1];
    __shared__ float s_lse[CLUSTERS ? HT : 1];
    __shared__ __align__(16) float s_q[MMA ? 1 : HT * D];
    __shared__ __align__(16) float s_p[MMA ? 1 : NW][MMA ? 1 : TILE * HT];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int units = a.Hkv * a.NG;

    int pos = 0, begin = 0, end = 1, b, u, t0, T_b, cum = 0, C = 1, rank = 0;
    if constexpr (CLUSTERS) {
        C = (int)cg::this_cluster().num_blocks();
        rank = (int)cg::this_cluster().block_rank();
        const int unit = blockIdx.x / C;
        b = unit / units;
        u = unit - b * units;
        T_b = tiles_of(a, b);
        if (T_b == 0) {  // no token, or a length out of range: the same in the whole cluster
            const int L = a.lens[b], h = u / a.NG, g0 = (u - h * a.NG) * HT, heads = min(HT, a.G - g0);
            const size_t at = (size_t)b * a.Hq + h * a.G + g0;
            const float fill = L == 0 ? 0.f : __int_as_float(0x7fc00000);
            if (rank == 0) {
                if (L != 0 && tid == 0) report(a.status, TV_ERR_INVALID_ARG);
                for (int i = tid; i < heads * D; i += DE_THREADS) Elem<T>::store(static_cast<T*>(a.out) + at * D + i, fill);
                if (a.lse && tid < heads) a.lse[at + tid] = L == 0 ? -__int_as_float(0x7f800000) : fill;
            }
            return;
        }
        t0 = (int)((int64_t)T_b * rank / C);
        pos = unit * a.cap_tiles + t0;  // where the scores go
        end = pos + (int)((int64_t)T_b * (rank + 1) / C) - t0;
    } else {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        // sequences without a token, and those whose length is out of range
        for (int x = blockIdx.x; x < a.B; x += gridDim.x) {
            const int L = a.lens[x];
            if (L > 0 && L <= a.max_len) continue;
            if (L != 0 && tid == 0) report(a.status, TV_ERR_INVALID_ARG);
            T* out = static_cast<T*>(a.out) + (size_t)x * a.Hq * D;
            const float fill = L == 0 ? 0.f : __int_as_float(0x7fc00000);
            for (int i = tid; i < a.Hq * D; i += DE_THREADS) Elem<T>::store(out + i, fill);
            if (a.lse)
                for (int i = tid; i < a.Hq; i += DE_THREADS)
                    a.lse[(size_t)x * a.Hq + i] = L == 0 ? -__int_as_float(0x7f800000) : fill;
        }
        find_start<NW>(a, units,
                       [&](int total) { return (int)min((int64_t)total, (int64_t)blockIdx.x * stretch(total, a.grid)); },
                       blockIdx.x == 0, &s_start, s_scan);
        const int total = s_start.total, per = stretch(total, a.grid);
        const int64_t begin64 = (int64_t)blockIdx.x * per;
        if (begin64 >= total) return;
        begin = pos = (int)begin64;
        end = (int)min((int64_t)total, begin64 + per);
        b = s_start.b;
        cum = s_start.cum;
        T_b = tiles_of(a, b);
        u = (pos - cum * units) / T_b;
        t0 = (pos - cum * units) - u * T_b;
    }

    unsigned char* ring = ring_all + warp * S::RING;
    const uint32_t ring_a = smem_u32(ring);
    const uint64_t policy = stream_policy();

    do {
        const int n = min(T_b - t0, end - pos);  // tiles of this piece (none for a CTA that a short sequence leaves over)
        const int L = a.lens[b];
        const int h = u / a.NG, g0 = (u - h * a.NG) * HT;
        const int heads = min(HT, a.G - g0);     // query heads of this unit
        const int32_t* table = a.c.table + (size_t)b * a.c.max_blocks;
        const T* q = static_cast<const T*>(a.q) + (size_t)b * a.q_stride + (size_t)(h * a.G + g0) * D;
        const char* kb = static_cast<const char*>(a.k) + (int64_t)h * a.c.head_stride;
        const char* vb = static_cast<const char*>(a.v) + (int64_t)h * a.c.head_stride;

        // the ring: tile i of the piece, for this warp i = warp, warp + NW, ...
        int bad = 0;
        auto offset_of = [&](int i) -> int64_t {  // lane's row of tile i, or -1
            const int t = (t0 + i) * TILE + lane % TILE;
            if (i >= n || t >= L) return -1;
            const int blk = t / a.c.block_size;
            const int id = table[blk];
            if (id < 0 || id >= a.c.num_blocks) {
                bad = 1;
                return -1;
            }
            return (int64_t)id * a.c.block_stride + (int64_t)(t - blk * a.c.block_size) * a.c.token_stride;
        };
        auto issue = [&](int slot, int64_t off) {
            const uint32_t dst = ring_a + slot * S::STAGE;
            static_assert(TILE * S::CH % 32 == 0, "a tile is whole warps of pieces");
#pragma unroll
            for (int j = 0; j < TILE * S::CH / 32; ++j) {
                const int x = j * 32 + lane, row = x / S::CH, ch = x - row * S::CH;
                const int64_t o = __shfl_sync(0xffffffffu, off, row);
                const int bytes = o < 0 ? 0 : 16;  // rows past the sequence are zeros
                const int64_t at = (o < 0 ? 0 : o) + ch * 16;
                cp_async16(dst + row * S::ROW + ch * 16, kb + at, bytes, policy);
                cp_async16(dst + TILE * S::ROW + row * S::ROW + ch * 16, vb + at, bytes, policy);
            }
        };
        // block ids of the first tiles and the queries: independent loads, all under way together
        int64_t off[S::STAGES];
#pragma unroll
        for (int e = 0; e < S::STAGES; ++e) off[e] = offset_of(warp + e * NW);
        // queries
        uint32_t qf[MMA ? NT : 1][MMA ? KS : 1][2];
        if constexpr (MMA) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int hd = j * 8 + lane / 4;
                const T* row = q + (size_t)hd * D + (lane % 4) * 2;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    qf[j][kk][0] = hd < heads ? *reinterpret_cast<const uint32_t*>(row + kk * 16) : 0u;
                    qf[j][kk][1] = hd < heads ? *reinterpret_cast<const uint32_t*>(row + kk * 16 + 8) : 0u;
                }
            }
        }

        int nxt = warp;  // next tile to request
#pragma unroll
        for (int e = 0; e < S::STAGES - 1; ++e) {
            if (nxt < n) issue(e, off[e]);
            cp_commit();
            nxt += NW;
        }
        int64_t off_next = off[S::STAGES - 1];
        if constexpr (!MMA) {
            for (int i = tid; i < HT * D; i += DE_THREADS) s_q[i] = i < heads * D ? reinterpret_cast<const float*>(q)[i] : 0.f;
            __syncthreads();
        }

        // running softmax: a lane of the matrix path has two heads per 8 (columns
        // 2 (lane % 4) and the next); on the fp32 path every lane has all HT
        constexpr int NM = MMA ? 2 * NT : HT;
        float m[NM], l[NM];
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
        float o[MMA ? NT * KS : HT][MMA ? 4 : DV];
#pragma unroll
        for (int i = 0; i < (MMA ? NT * KS : HT); ++i)
#pragma unroll
            for (int e = 0; e < (MMA ? 4 : DV); ++e) o[i][e] = 0.f;

        int slot = 0;
        for (int i = warp; i < n; i += NW) {
            cp_wait<S::STAGES - 2>();
            __syncwarp();
            {  // the slot that the previous step read is free
                int free_slot = slot + S::STAGES - 1;
                if (free_slot >= S::STAGES) free_slot -= S::STAGES;
                if (nxt < n) issue(free_slot, off_next);
                cp_commit();
                nxt += NW;
                off_next = offset_of(nxt);
            }
            const uint32_t kt = ring_a + slot * S::STAGE, vt = kt + TILE * S::ROW;
            const int tok = (t0 + i) * TILE;
            float* sc = a.weights ? a.scores + ((size_t)(pos + i) * TILE) * a.GS : nullptr;
            if constexpr (MMA) {
                float c[NT][4], c2[NT][4];  // two chains of products
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[j][e] = c2[j][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk) {
                    uint32_t f[4];
                    ldsm4(f, kt + (lane % 16) * S::ROW + (kk * 2 + lane / 16) * 16);
#pragma unroll
                    for (int j = 0; j < NT; ++j) Mma<T>::run(kk & 1 ? c2[j] : c[j], f, qf[j][kk][0], qf[j][kk][1]);
                }
                const int r0 = lane / 4;
                const bool in0 = tok + r0 < L, in1 = tok + r0 + 8 < L;
                bool grew = false;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        c[j][e] = in0 ? (c[j][e] + c2[j][e]) * a.scale_log2 : -INFINITY;
                        c[j][2 + e] = in1 ? (c[j][2 + e] + c2[j][2 + e]) * a.scale_log2 : -INFINITY;
                        grew |= fmaxf(c[j][e], c[j][2 + e]) > m[2 * j + e] + REF_MOVES;
                    }
                    const int hd = j * 8 + (lane % 4) * 2;
                    if (sc) {
                        if (!(a.GS & 1)) {  // pairs are aligned; one may reach past `heads`, inside the GS of a token
                            if (in0 && hd < heads) *reinterpret_cast<float2*>(sc + r0 * a.GS + hd) = make_float2(c[j][0], c[j][1]);
                            if (in1 && hd < heads)
                                *reinterpret_cast<float2*>(sc + (r0 + 8) * a.GS + hd) = make_float2(c[j][2], c[j][3]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                if (in0 && hd + e < heads) sc[r0 * a.GS + hd + e] = c[j][e];
                                if (in1 && hd + e < heads) sc[(r0 + 8) * a.GS + hd + e] = c[j][2 + e];
                            }
                        }
                    }
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int k = 0; k < NM; ++k) {
                        const int j = k / 2, e = k % 2;
                        float x = fmaxf(c[j][e], c[j][2 + e]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        x = fmaxf(m[k], x - REF_BELOW);
                        const float corr = x == -INFINITY ? 1.f : ex2(m[k] - x);
                        m[k] = x;
                        l[k] *= corr;
#pragma unroll
                        for (int d = 0; d < KS; ++d) {
                            o[j * KS + d][e] *= corr;
                            o[j * KS + d][2 + e] *= corr;
                        }
                    }
                }
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mu = m[2 * j + e] == -INFINITY ? 0.f : m[2 * j + e];
                        c[j][e] = ex2(c[j][e] - mu);
                        c[j][2 + e] = ex2(c[j][2 + e] - mu);
                        l[2 * j + e] += c[j][e] + c[j][2 + e];
                    }
                    Mma<T>::split(c[j][0], c[j][1], ph[j][0], pl[j][0]);
                    Mma<T>::split(c[j][2], c[j][3], ph[j][1], pl[j][1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ph[j][e] = movm(ph[j][e]);
                        pl[j][e] = movm(pl[j][e]);
                    }
                }
#pragma unroll
                for (int d = 0; d < KS; ++d) {
                    uint32_t f[4];
                    ldsm4t(f, vt + ((lane % 8) + (lane / 16) * 8) * S::ROW + (d * 2 + (lane / 8) % 2) * 16);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        Mma<T>::run(o[j * KS + d], f, ph[j][0], ph[j][1]);
                        Mma<T>::run(o[j * KS + d], f, pl[j][0], pl[j][1]);
                    }
                }
            } else {
                const unsigned char* kr = ring + slot * S::STAGE;
                const unsigned char* vr = kr + TILE * S::ROW;
                const int tk = lane / 2, half = lane % 2;
                float acc[HT];
#pragma unroll
                for (int g = 0; g < HT; ++g) acc[g] = 0.f;
#pragma unroll 4
                for (int x = 0; x < D / 8; ++x) {
                    const float4 kv = *reinterpret_cast<const float4*>(kr + tk * S::ROW + (2 * x + half) * 16);
#pragma unroll
                    for (int g = 0; g < HT; ++g) {
                        const float4 qv = *reinterpret_cast<const float4*>(&s_q[g * D + (2 * x + half) * 4]);
                        acc[g] = fmaf(kv.x, qv.x, acc[g]);
                        acc[g] = fmaf(kv.y, qv.y, acc[g]);
                        acc[g] = fmaf(kv.z, qv.z, acc[g]);
                        acc[g] = fmaf(kv.w, qv.w, acc[g]);
                    }
                }
                const bool in = tok + tk < L;
                bool grew = false;
                float corr[HT];
#pragma unroll
                for (int g = 0; g < HT; ++g) {
                    float x = acc[g] + __shfl_xor_sync(0xffffffffu, acc[g], 1);
                    x = in ? x * a.scale_log2 : -INFINITY;
                    if (sc && half == 0 && in && g < heads) sc[tk * a.GS + g] = x;
                    float y = x;
#pragma unroll
                    for (int d = 2; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                    const float mn = fmaxf(m[g], y);
                    const float mu = mn == -INFINITY ? 0.f : mn;
                    corr[g] = ex2(m[g] - mu);
                    grew |= mn != m[g];
                    m[g] = mn;
                    const float p = ex2(x - mu);
                    l[g] = l[g] * corr[g] + (half ? 0.f : p);
                    if (half == 0) s_p[warp][tk * HT + g] = p;
                }
                __syncwarp();
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int g = 0; g < HT; ++g)
#pragma unroll
                        for (int e = 0; e < DV; ++e) o[g][e] *= corr[g];
                }
#pragma unroll 4
                for (int t = 0; t < TILE; ++t) {
                    float vv[DV];
#pragma unroll
                    for (int e = 0; e < DV; ++e) vv[e] = reinterpret_cast<const float*>(vr + t * S::ROW)[lane + 32 * e];
                    float pp[HT];
#pragma unroll
                    for (int g = 0; g < HT; g += 4)
                        *reinterpret_cast<float4*>(pp + g) = *reinterpret_cast<const float4*>(&s_p[warp][t * HT + g]);
#pragma unroll
                    for (int g = 0; g < HT; ++g) {
#pragma unroll
                        for (int e = 0; e < DV; ++e) o[g][e] = fmaf(pp[g], vv[e], o[g][e]);
                    }
                }
            }
            __syncwarp();
            if (++slot == S::STAGES) slot = 0;
        }
        cp_wait<0>();
        __syncwarp();

        // the warps' parts: common maximum, then sums (in warp order) through the rings
#pragma unroll
        for (int k = 0; k < NM; ++k) {
#pragma unroll
            for (int d = MMA ? 4 : 1; d < 32; d <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], d);
            const int hd = MMA ? (k / 2) * 8 + (lane % 4) * 2 + k % 2 : k;
            if (MMA ? lane < 4 : lane == 0) {
                s_m[warp][hd] = m[k];
                s_l[warp][hd] = l[k];
            }
        }
        int any_bad = __syncthreads_or(bad);
        constexpr int OROW = D + 4;
        static_assert(HT * OROW * 4 <= S::RING, "a warp's outputs fit its ring");
        float* so = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int k = 0; k < NM; ++k) {
            const int hd = MMA ? (k / 2) * 8 + (lane % 4) * 2 + k % 2 : k;
            float M = s_m[0][hd];
#pragma unroll
            for (int w = 1; w < NW; ++w) M = fmaxf(M, s_m[w][hd]);
            const float f = ex2(m[k] - (M == -INFINITY ? 0.f : M));
            if constexpr (MMA) {
#pragma unroll
                for (int d = 0; d < KS; ++d) {
                    so[hd * OROW + d * 16 + lane / 4] = o[(k / 2) * KS + d][k % 2] * f;
                    so[hd * OROW + d * 16 + lane / 4 + 8] = o[(k / 2) * KS + d][2 + k % 2] * f;
                }
            } else {
#pragma unroll
                for (int e = 0; e < DV; ++e) so[hd * OROW + lane + 32 * e] = o[k][e] * f;
            }
        }
        __syncthreads();
        const bool whole = !CLUSTERS && n == T_b;
        const int part = 2 * blockIdx.x + (pos == begin ? 0 : 1);
        if (any_bad && tid == 0) report(a.status, TV_ERR_BLOCK_TABLE);
        float* joint = reinterpret_cast<float*>(ring_all) + HT * OROW;  // clusters: this CTA's sums, behind warp 0's
        static_assert(2 * HT * OROW * 4 <= S::RING, "a warp's outputs and the CTA's fit its ring");
        for (int x = tid; x < heads * (D / 4); x += DE_THREADS) {
            const int hd = x / (D / 4), d = (x - hd * (D / 4)) * 4;
            float M = s_m[0][hd], sum = 0.f;
#pragma unroll
            for (int w = 1; w < NW; ++w) M = fmaxf(M, s_m[w][hd]);
            const float mu = M == -INFINITY ? 0.f : M;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                sum += s_l[w][hd] * ex2(s_m[w][hd] - mu);
                const float4 y = *reinterpret_cast<const float4*>(ring_all + w * S::RING + (hd * OROW + d) * 4);
                r.x += y.x;
                r.y += y.y;
                r.z += y.z;
                r.w += y.w;
            }
            if (whole) {
                float inv = sum == 0.f ? 0.f : 1.f / sum;
                if (any_bad) inv = __int_as_float(0x7fc00000);
                T* out = static_cast<T*>(a.out) + ((size_t)b * a.Hq + h * a.G + g0 + hd) * D + d;
                Elem<T>::store(out, r.x * inv);
                Elem<T>::store(out + 1, r.y * inv);
                Elem<T>::store(out + 2, r.z * inv);
                Elem<T>::store(out + 3, r.w * inv);
                if (d == 0) {
                    const size_t at = (size_t)b * a.Hq + h * a.G + g0 + hd;
                    const float l2 = sum == 0.f ? -INFINITY : M + log2f(sum);
                    if (a.lse) a.lse[at] = any_bad ? __int_as_float(0x7fc00000) : l2 * LN2;
                    // +inf marks a head whose weights stay as they were
                    if (a.weights) a.lse2[at] = any_bad ? INFINITY : l2;
                }
            } else if constexpr (CLUSTERS) {
                *reinterpret_cast<float4*>(joint + hd * OROW + d) = r;
                if (d == 0) s_ml[hd] = make_float2(M, any_bad ? BAD_SUM : sum);
            } else {
                *reinterpret_cast<float4*>(a.part_o + ((size_t)part * HT + hd) * D + d) = r;
                if (d == 0) a.part_ml[(size_t)part * HT + hd] = make_float2(M, any_bad ? BAD_SUM : sum);
            }
        }
        if constexpr (CLUSTERS) {
            cg::cluster_group cluster = cg::this_cluster();
            // the old sum of this thread's first token is on its way during the join
            float* w = a.weights ? a.weights + ((size_t)b * a.Hkv + h) * a.weight_stride : nullptr;
            const int first_t = t0 * TILE + tid, end_t = min(L, (t0 + n) * TILE);
            float old = w && first_t < end_t ? w[first_t] : 0.f;
            cluster.sync();
            const size_t at = (size_t)b * a.Hq + h * a.G + g0;
            // every head's common reference, sum and flag, in rank order
            if (tid < heads) {
                float M = -INFINITY, sum = 0.f;
                bool flag = false;
                for (int c = 0; c < C; ++c) {
                    const float2 ml = *cluster.map_shared_rank(&s_ml[tid], c);
                    M = fmaxf(M, ml.x);
                    flag |= ml.y == BAD_SUM;
                }
                for (int c = 0; c < C; ++c) {
                    const float2 ml = *cluster.map_shared_rank(&s_ml[tid], c);
                    sum += ml.y * ex2(ml.x - (M == -INFINITY ? 0.f : M));
                }
                const float l2 = sum == 0.f ? -INFINITY : M + log2f(sum), nan = __int_as_float(0x7fc00000);
                s_m[0][tid] = M == -INFINITY ? 0.f : M;
                s_l[0][tid] = flag ? nan : sum == 0.f ? 0.f : 1.f / sum;
                // a head without a finite score gets no weight: exp2(s - inf) = 0
                s_lse[tid] = l2 == -INFINITY ? INFINITY : l2;
                if (a.lse && rank == 0) a.lse[at + tid] = flag ? nan : l2 * LN2;
                any_bad = flag;
            }
            any_bad = __syncthreads_or(any_bad);
            for (int x = rank * DE_THREADS + tid; x < heads * (D / 4); x += C * DE_THREADS) {
                const int hd = x / (D / 4), d = (x - hd * (D / 4)) * 4;
                const float mu = s_m[0][hd], inv = s_l[0][hd];
                float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c = 0; c < C; ++c) {
                    const float f = ex2(cluster.map_shared_rank(&s_ml[hd], c)->x - mu);
                    const float4 y = *reinterpret_cast<const float4*>(cluster.map_shared_rank(joint + hd * OROW + d, c));
                    r.x += y.x * f;
                    r.y += y.y * f;
                    r.z += y.z * f;
                    r.w += y.w * f;
                }
                T* out = static_cast<T*>(a.out) + (at + hd) * D + d;
                Elem<T>::store(out, r.x * inv);
                Elem<T>::store(out + 1, r.y * inv);
                Elem<T>::store(out + 2, r.z * inv);
                Elem<T>::store(out + 3, r.w * inv);
            }
            __syncwarp();
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this CTA has read its peers' parts
            if (w && !any_bad) {  // one unit per KV head here; this CTA wrote these scores itself
                const float* scores = a.scores + (size_t)(pos - t0) * TILE * a.GS;
                for (int t = first_t; t < end_t; t += DE_THREADS) {
                    float sum = 0.f;
                    for (int g = 0; g < heads; ++g) sum += ex2(scores[(size_t)t * a.GS + g] - s_lse[g]);
                    w[t] = (t == first_t ? old : w[t]) + sum;
                }
            }
            __syncwarp();
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // and they this CTA's
            return;
        }
        __syncthreads();  // the rings and the shared values are free for the next piece

        pos += n;
        t0 = 0;
        if (++u == units) {
            u = 0;
            cum += T_b;
            if (pos < end) do T_b = tiles_of(a, ++b); while (T_b == 0);
        }
    } while (pos < end);
}

// Where a unit's tiles lie on the line and which stretches cover them.
struct Pieces {
    int c0, c1, per, first;  // stretches c0 .. c1; first: the unit's first tile
    __device__ __forceinline__ int slot(int c) const { return 2 * c + (c == c0 && c * per != first ? 1 : 0); }
};
__device__ __forceinline__ Pieces pieces_of(int first, int tiles, int per) {
    Pieces p;
    p.first = first;
    p.per = per;
    p.c0 = first / per;
    p.c1 = (first + tiles - 1) / per;
    return p;
}

// The sequence that holds tile `pos` of the line (the last b whose tiles begin at or before it).
__device__ __forceinline__ int find_seq(const int32_t* cum, int B, int pos, int units) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cum[mid] * units <= pos) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

constexpr int JO_THREADS = 128;
constexpr int JO_UN = 4;      // rows of a thread that are loaded ahead
constexpr int CUM_MAX = 512;  // sequences whose tile counts a join CTA adds up itself
constexpr int WT_UN = 4;  // tokens of a thread whose scores are loaded at once

// Joins the pieces of the heads that several CTAs share, and adds the
// weights.  The first `wblocks` blocks share the line of (sequence, KV head, tile) for
// the weights.  The others are one per query head of a unit: by_unit, of every unit;
// else (more units than stretches) of the unit in which stretch y begins, if
// that stretch is the unit's second.
template <typename T, int D, int HT>
__global__ void __launch_bounds__(JO_THREADS) decode_join_kernel(const __grid_constant__ DecodeArgs a, int wblocks,
                                                                bool by_unit) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int units = a.Hkv * a.NG;
    __shared__ float s_red[2][JO_THREADS / 32];
    __shared__ float4 s_o[JO_THREADS];
    __shared__ __align__(16) float s_lse[128];
    // The tiles before each sequence: of a small batch from the lengths, while the first kernel still runs;
    // of a large one as that kernel wrote them.
    __shared__ int32_t s_cum[CUM_MAX + 1];
    __shared__ int s_scan[JO_THREADS / 32];
    const int32_t* cum = a.cum;
    if (a.B <= CUM_MAX) {
        constexpr int RUN = CUM_MAX / JO_THREADS;
        int t[RUN], sum = 0;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            t[i] = tid * RUN + i < a.B ? tiles_of(a, tid * RUN + i) : 0;
            sum += t[i];
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int before = inc - sum;
#pragma unroll
        for (int w = 0; w < JO_THREADS / 32; ++w)
            if (w < warp) before += s_scan[w];
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            if (tid * RUN + i <= a.B) s_cum[tid * RUN + i] = before;
            before += t[i];
        }
        if (tid == JO_THREADS - 1 && a.B == CUM_MAX) s_cum[CUM_MAX] = before;
        __syncthreads();
        cum = s_cum;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int all = cum[a.B], total = all * units;
    if (total == 0) return;
    const int per = stretch(total, a.grid);
    if ((int)blockIdx.x >= wblocks) {
        const int x = blockIdx.x - wblocks, y = x / a.GS, hd = x - y * a.GS;
        int b, u, T_b, first;
        if (by_unit) {
            b = y / units;
            u = y - b * units;
            T_b = cum[b + 1] - cum[b];
            first = cum[b] * units + u * T_b;
            if (T_b == 0 || first / per == (first + T_b - 1) / per) return;  // empty, or one stretch had it whole
        } else {
            if (y == 0 || (int64_t)y * per >= total) return;
            const int pos = y * per;
            b = find_seq(cum, a.B, pos, units);
            const int base = cum[b] * units;
            T_b = cum[b + 1] - cum[b];
            u = (pos - base) / T_b;
            first = base + u * T_b;
            if (pos == first || pos - per > first) return;  // the unit's first stretch, or a later one than its second
        }
        const int h = u / a.NG, g0 = (u - h * a.NG) * HT;
        if (g0 + hd >= a.G) return;
        const Pieces p = pieces_of(first, T_b, per);
        constexpr int Q = D / 4, GR = JO_THREADS / Q;  // lanes of a row, rows at once
        const int gr = tid / Q, d = tid - gr * Q;
        // the first rows are on their way during the maximum
        float4 row[JO_UN];
#pragma unroll
        for (int k = 0; k < JO_UN; ++k) {
            const int i = p.c0 + gr + k * GR;
            row[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (gr < GR && i <= p.c1)
                row[k] = *reinterpret_cast<const float4*>(a.part_o + ((size_t)p.slot(i) * HT + hd) * D + d * 4);
        }
        // maximum and sum over the pieces
        float M = -INFINITY, bad = 0.f;
        for (int i = p.c0 + tid; i <= p.c1; i += JO_THREADS) {
            const float2 ml = a.part_ml[(size_t)p.slot(i) * HT + hd];
            M = fmaxf(M, ml.x);
            if (ml.y == BAD_SUM) bad = 1.f;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
            bad = fmaxf(bad, __shfl_xor_sync(0xffffffffu, bad, d));
        }
        if (lane == 0) {
            s_red[0][warp] = M;
            s_red[1][warp] = bad;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < JO_THREADS / 32; ++w) {
            M = fmaxf(M, s_red[0][w]);
            bad = fmaxf(bad, s_red[1][w]);
        }
        const float mu = M == -INFINITY ? 0.f : M;
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
        auto add = [&](int i, const float4& y) {
            const float2 ml = a.part_ml[(size_t)p.slot(i) * HT + hd];
            const float f = ex2(ml.x - mu);
            sum += ml.y * f;
            r.x += y.x * f;
            r.y += y.y * f;
            r.z += y.z * f;
            r.w += y.w * f;
        };
        if (gr < GR) {
#pragma unroll
            for (int k = 0; k < JO_UN; ++k)
                if (p.c0 + gr + k * GR <= p.c1) add(p.c0 + gr + k * GR, row[k]);
            for (int i = p.c0 + gr + JO_UN * GR; i <= p.c1; i += GR)
                add(i, *reinterpret_cast<const float4*>(a.part_o + ((size_t)p.slot(i) * HT + hd) * D + d * 4));
        }
        __shared__ float s_sum[JO_THREADS];
        s_o[tid] = r;
        s_sum[tid] = sum;
        __syncthreads();
        if (gr == 0) {
#pragma unroll
            for (int g = 1; g < GR; ++g) {
                const float4 y = s_o[g * Q + d];
                r.x += y.x;
                r.y += y.y;
                r.z += y.z;
                r.w += y.w;
                sum += s_sum[g * Q + d];
            }
            float inv = sum == 0.f ? 0.f : 1.f / sum;
            if (bad != 0.f) inv = __int_as_float(0x7fc00000);
            const size_t at = (size_t)b * a.Hq + h * a.G + g0 + hd;
            T* out = static_cast<T*>(a.out) + at * D + d * 4;
            Elem<T>::store(out, r.x * inv);
            Elem<T>::store(out + 1, r.y * inv);
            Elem<T>::store(out + 2, r.z * inv);
            Elem<T>::store(out + 3, r.w * inv);
            if (d == 0 && a.lse)
                a.lse[at] = bad != 0.f ? __int_as_float(0x7fc00000) : sum == 0.f ? -INFINITY : (M + log2f(sum)) * LN2;
        }
        return;
    }
    // weights: an equal stretch of (sequence, KV head, tile) for every block
    const int wb = blockIdx.x;
    const int wtotal = all * a.Hkv, wper = (wtotal + wblocks - 1) / wblocks;
    if ((int64_t)wb * wper >= wtotal) return;
    int pos = wb * wper;
    const int end = min(wtotal, pos + wper);
    int b = find_seq(cum, a.B, pos, a.Hkv);
    while (pos < end) {
        const int T_b = cum[b + 1] - cum[b];
        const int base = cum[b] * a.Hkv, h = (pos - base) / T_b, t0 = pos - base - h * T_b;
        const int n = min(T_b - t0, end - pos);
        // log-sum-exp of the KV head's query heads, a warp each
        int bad_any = 0;
        __syncthreads();
        for (int g = warp; g < a.G; g += JO_THREADS / 32) {
            const int k = g / HT, hd = g - k * HT, first = cum[b] * units + (h * a.NG + k) * T_b;
            const Pieces p = pieces_of(first, T_b, per);
            float x;
            if (p.c0 == p.c1) {
                x = a.lse2[(size_t)b * a.Hq + h * a.G + g];
            } else {
                float M = -INFINITY, sum = 0.f, bad = 0.f;
                for (int i = p.c0 + lane; i <= p.c1; i += 32) {
                    const float2 ml = a.part_ml[(size_t)p.slot(i) * HT + hd];
                    M = fmaxf(M, ml.x);
                    if (ml.y == BAD_SUM) bad = 1.f;
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) {
                    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
                    bad = fmaxf(bad, __shfl_xor_sync(0xffffffffu, bad, d));
                }
                const float mu = M == -INFINITY ? 0.f : M;
                for (int i = p.c0 + lane; i <= p.c1; i += 32) {
                    const float2 ml = a.part_ml[(size_t)p.slot(i) * HT + hd];
                    sum += ml.y * ex2(ml.x - mu);
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                x = bad != 0.f ? INFINITY : sum == 0.f ? -INFINITY : M + log2f(sum);
            }
            bad_any |= x == INFINITY;
            // a head without a finite score gets no weight: exp2(s - inf) = 0
            if (lane == 0) s_lse[g] = x == -INFINITY ? INFINITY : x;
        }
        const int L = a.lens[b];
        float* w = a.weights + ((size_t)b * a.Hkv + h) * a.weight_stride;
        // scores of a token lie side by side: GS for each of the KV head's NG units
        const float* scores = a.scores + ((size_t)cum[b] * units + (size_t)h * a.NG * T_b) * TILE * a.GS;
        const size_t unit_scores = (size_t)T_b * TILE * a.GS;
        auto weight_of = [&](int t) {
            float sum = 0.f;
            for (int k = 0; k < a.NG; ++k) {
                const float* sc = scores + k * unit_scores + (size_t)t * a.GS;
                const float* lse = s_lse + k * HT;
                const int heads = min(HT, a.G - k * HT);
                if (a.GS % 4 == 0) {
#pragma unroll
                    for (int g = 0; g < HT; g += 4) {
                        if (g + 4 <= heads) {
                            const float4 y = *reinterpret_cast<const float4*>(sc + g);
                            const float4 z = *reinterpret_cast<const float4*>(lse + g);
                            sum += (ex2(y.x - z.x) + ex2(y.y - z.y)) + (ex2(y.z - z.z) + ex2(y.w - z.w));
                        } else {
                            for (int e = g; e < heads; ++e) sum += ex2(sc[e] - lse[e]);
                            break;
                        }
                    }
                } else {
                    for (int g = 0; g < heads; ++g) sum += ex2(sc[g] - lse[g]);
                }
            }
            return sum;
        };
        if (!__syncthreads_or(bad_any)) {
            const int t1 = min(L, (t0 + n) * TILE);
            for (int x = t0 * TILE + tid; x < t1; x += WT_UN * JO_THREADS) {
                float sum[WT_UN], old[WT_UN];
#pragma unroll
                for (int e = 0; e < WT_UN; ++e) {
                    const int t = x + e * JO_THREADS;
                    sum[e] = old[e] = 0.f;
                    if (t < t1) {
                        old[e] = w[t];
                        sum[e] = weight_of(t);
                    }
                }
#pragma unroll
                for (int e = 0; e < WT_UN; ++e)
                    if (x + e * JO_THREADS < t1) w[x + e * JO_THREADS] = old[e] + sum[e];
            }
        }
        pos += n;
        while (pos < end && pos >= cum[b + 1] * a.Hkv) ++b;
    }
}

template <typename T, int D, int HT>
cudaError_t launch(const DecodeArgs& a, const DecodePlan& p, cudaStream_t st) {
    constexpr int threads = Shape<T, D>::NW * 32, smem = Shape<T, D>::NW * Shape<T, D>::RING;
    if (p.cluster) {
        auto kern = decode_kernel<T, D, HT, true>;
        static SmemLimit limit;  // one size for every call of this kernel
        cudaError_t e = limit.allow((const void*)kern, smem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(p.grid);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = p.cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, a);
    }
    auto kern = decode_kernel<T, D, HT, false>;
    static SmemLimit limit;
    cudaError_t e = limit.allow((const void*)kern, smem);
    if (e != cudaSuccess) return e;
    kern<<<p.grid, threads, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int wblocks = a.weights ? 4 * p.grid : 0;
    cudaLaunchConfig_t cfg = {};
    const int64_t all_units = (int64_t)a.B * a.Hkv * a.NG;
    const bool by_unit = all_units <= p.grid;
    cfg.gridDim = dim3(wblocks + (by_unit ? (int)all_units : p.grid) * a.GS);
    cfg.blockDim = dim3(JO_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_join_kernel<T, D, HT>, a, wblocks, by_unit);
}

template <typename T, int HT>
cudaError_t by_dim(const DecodeArgs& a, const DecodePlan& p, cudaStream_t st) {
    switch (a.D) {
        case 64: return launch<T, 64, HT>(a, p, st);
        case 96: return launch<T, 96, HT>(a, p, st);
        case 128: return launch<T, 128, HT>(a, p, st);
        default:
            if constexpr (HT <= 8) return launch<T, 256, HT>(a, p, st);
            return cudaErrorInvalidValue;
    }
}

}  // namespace

void decode_plan(int dtype, int B, int Hkv, int G, int D, int max_len, bool weights, int sms, DecodePlan* p) {
    const int es = dtype == TV_F32 ? 4 : 2;
    if (dtype == TV_F32) p->HT = G <= 4 ? 4 : 8;
    else p->HT = G <= 8 || D > 128 ? 8 : 16;
    p->NG = (G + p->HT - 1) / p->HT;
    p->GS = G < p->HT ? G : p->HT;
    // as in Shape
    const int ring = (es == 2 ? 3 : 2) * 2 * TILE * (D * es + (es == 2 ? 16 : 32));
    const int fit = 210 * 1024 / ring, warps = es == 2 ? 4 : fit < 8 ? fit : 8;
    p->smem = ring * warps;
    const int fixed = 4096 + (es == 4 ? p->HT * D * 4 + warps * TILE * p->HT * 4 : 0);  // static and reserved shared memory
    int per_sm = (228 * 1024) / (p->smem + fixed);
    if (per_sm < 1) per_sm = 1;
    if (per_sm > 4) per_sm = 4;
    const int64_t units = (int64_t)B * Hkv * p->NG, cap_tiles = (max_len + TILE - 1) / TILE, tiles = units * cap_tiles;
    // Clusters of up to 8 CTAs per unit, down to 4 tiles (one per warp) for each, where that is short
    // work (8 tiles per CTA; 1,024 tokens of one sequence with 8 KV heads: 6.7 us, by stretches 8.4) or
    // fills most of the GPU (up to 32 tiles; 4 x 2,048 tokens 11.4 us against 14.6, 64 x 512 32.3
    // against 34.1).  Past that the equal stretches win: they use every SM (one sequence of 4,096: 9.9
    // against 11.8) and do not depend on how long each sequence of a batch is.  Clusters of 16 lost
    // to 8 at 1,024 tokens (7.7 us).  Weights over several units of a KV head need the second kernel.
    p->cluster = 0;
    if (!weights || p->NG == 1) {
        int c = 1;
        while (c < 8 && c * 4 < cap_tiles && units * c * 2 <= (int64_t)per_sm * sms) c *= 2;
        if (cap_tiles <= c * 8 || (cap_tiles <= c * 32 && units * c * 4 >= 3 * (int64_t)sms)) {
            p->cluster = c;
            p->grid = (int)(units * c);
            return;
        }
    }
    int64_t grid = (tiles + MIN_TILES - 1) / MIN_TILES;
    if (grid > (int64_t)per_sm * sms) grid = (int64_t)per_sm * sms;
    if (grid < 1) grid = 1;
    p->grid = (int)grid;
}

cudaError_t launch_decode(const DecodeArgs& a, int dtype, const DecodePlan& p, cudaStream_t st) {
    if (dtype == TV_BF16) return p.HT == 8 ? by_dim<__nv_bfloat16, 8>(a, p, st) : by_dim<__nv_bfloat16, 16>(a, p, st);
    if (dtype == TV_F16) return p.HT == 8 ? by_dim<__half, 8>(a, p, st) : by_dim<__half, 16>(a, p, st);
    return p.HT == 4 ? by_dim<float, 4>(a, p, st) : by_dim<float, 8>(a, p, st);
}

}  // namespace tv
