// rotary.cu -- tv_rotary_write: a step's queries and keys are rotated by their
// positions, keys and values are written into the paged cache.
//
// Pair i of a head (elements i and i + R/2, or 2i and 2i + 1) turns by
// pos[axis(i)] * inv_freq[i]:
//     x' = x cos - y sin,   y' = x sin + y cos.
// The product is formed in fp64 and reduced to a fraction of a turn there: at
// position 131,072 an fp32 product is off by up to 2^-8 of a radian, the fp64
// one by less than 2^-35.  What is left lies in [-1/2, 1/2] turns and goes to
// fp32 sincospi.  The cosines and sines of a node serve all of its heads.
//
// One CTA per node.  Every thread's first loads are under way while one thread
// looks up where the rows go and the first R/2 threads form the angles.
//
// Bound: HBM (each row is read once and written once): a 16,384-token prompt of 32 + 8 + 8
// heads (403 MB) takes 67 us, 92 % of the copy bandwidth.  That needed few
// instructions: with a division per 16-byte piece and the cosines read from
// shared memory for each, it took 107 to 123 us.  A small call is launch and
// three dependent loads (4 us for one 64-node tree; 5 with its parents read from
// global memory, one after the other).
#include "kernels.h"
#include "tv_common.cuh"

namespace tv {
namespace {

constexpr int RO_THREADS = 128;

// 16 bytes as fp32 values, and back
template <typename T> struct Pack;
template <> struct Pack<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4& u, float* f) {
        f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Pack<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& u, float* f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Pack<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& u, float* f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
    static __device__ __forceinline__ uint4 put(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Depth of node j (steps to the root), or -1 when its path is malformed; parents in shared memory.
__device__ __forceinline__ int node_depth(const int32_t* parent, int j) {
    int depth = 0;
    while (j > 0) {
        const int p = parent[j];
        if (p < 0 || p >= j) return -1;
        j = p;
        ++depth;
    }
    return parent[0] == -1 ? depth : -1;
}

// TREE: depths from a parent array.  A kernel of its own: with a branch for it, the first loads of
// a prompt's rows came later (79 us against 68 for 16,384 tokens).
template <typename T, bool INTER, bool TREE>
__global__ void __launch_bounds__(RO_THREADS) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    constexpr int PN = Pack<T>::N;
    constexpr int NF = INTER ? PN / 2 : PN;  // frequencies of a thread's pieces
    // Heads of a thread that are loaded at once (the first before the angles are known): 32 + 8 heads
    // of 128 are five of one piece (interleaved; 64 ragged trees took 7.2 us with three, 6.7 with
    // five) or three of two pieces.
    constexpr int RO_UN = INTER ? 5 : 3;
    __shared__ __align__(16) float s_cos[128], s_sin[128];
    __shared__ long long s_off;
    __shared__ int s_bad;
    extern __shared__ int32_t s_parent[];  // with a parent array: N of them
    const int tid = threadIdx.x, b = blockIdx.x / a.N, j = blockIdx.x - b * a.N;
    bool bad_count;
    const int n = seq_nodes(a.counts, b, a.N, bad_count);
    if (j >= n) return;
    const int L = a.prefix_lens[b];
    if constexpr (TREE)  // the parents that a path from node j can meet
        for (int i = tid; i <= j; i += RO_THREADS) s_parent[i] = a.parent[(size_t)b * a.N + i];
    const size_t node = (size_t)b * a.N + j;
    // A thread keeps to one place of the rows: piece i (and i + Rp / 2), of the heads
    // g, g + groups, ...: the query heads, then the key heads.
    const int Dp = a.D / PN, Rp = a.rot / PN;  // 16-byte pieces of a row; rotated pieces
    const int units = INTER ? Dp : Dp - Rp / 2, groups = RO_THREADS / units;
    const int g = tid / units, i = tid - g * units;
    const bool turns_here = i < (INTER ? Rp : Rp / 2);
    const int at = INTER || turns_here ? i : i + Rp / 2;  // past the rotated part: one piece
    const int qh = a.q ? a.Hq : 0, heads = g < groups ? qh + a.Hkv : 0;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + node * a.q_stride) + at;
    const uint4* k = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + node * a.k_stride) + at;
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + node * a.v_stride);
    auto load = [&](int h, uint4& u, uint4& w) {
        const uint4* src = h < qh ? q + h * Dp : k + (h - qh) * Dp;
        u = src[0];
        if (!INTER && turns_here) w = src[Rp / 2];
    };
    uint4 u[RO_UN], w[RO_UN], vv = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < RO_UN; ++e)
        if (g + e * groups < heads) load(g + e * groups, u[e], w[e]);
    if (tid < a.Hkv * Dp) vv = v[tid];

    if (tid == RO_THREADS - 1) {  // where the rows go
        int bad = 0;
        long long off = 0;
        if (bad_count || L < 0 || (long long)L + n > (long long)a.c.max_blocks * a.c.block_size) {
            bad = TV_ERR_INVALID_ARG;
        } else {
            const int t = L + j, blk = t / a.c.block_size;
            const int id = a.c.table[(size_t)b * a.c.max_blocks + blk];
            if (id < 0 || id >= a.c.num_blocks) bad = TV_ERR_BLOCK_TABLE;
            else off = (long long)id * a.c.block_stride + (long long)(t - blk * a.c.block_size) * a.c.token_stride;
        }
        s_off = off;
        s_bad = bad;
    }
    int depth = j;
    if constexpr (TREE) {
        __syncthreads();
        depth = node_depth(s_parent, j);
    }
    if (tid < a.rot / 2) {
        const int ax = a.axis_of_pair[tid];
        double pos;
        if (a.positions) pos = (double)a.positions[((size_t)ax * a.B + b) * a.N + j];
        else pos = (double)(a.position_base ? a.position_base[b] : L) + (double)depth;
        const double turns = pos * (double)a.inv_freq[tid] * 0.15915494309189533577;
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
        s_cos[tid] = cs;
        s_sin[tid] = sn;
    }
    __syncthreads();
    const int bad = s_bad ? s_bad : depth < 0 ? TV_ERR_TREE : 0;
    uint4* qo = reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + node * (size_t)a.Hq * a.D);
    if (bad) {  // NaN queries, nothing else
        if (tid == 0) report(a.status, bad);
        float x[PN];
#pragma unroll
        for (int e = 0; e < PN; ++e) x[e] = __int_as_float(0x7fc00000);
        for (int y = tid; y < qh * Dp; y += RO_THREADS) qo[y] = Pack<T>::put(x);
        return;
    }
    char* ck = static_cast<char*>(a.cache_k) + s_off;
    char* cv = static_cast<char*>(a.cache_v) + s_off;
    float cs[NF], sn[NF];
    if (turns_here) {
#pragma unroll
        for (int e = 0; e < NF; ++e) {
            cs[e] = s_cos[i * NF + e];
            sn[e] = s_sin[i * NF + e];
        }
    }
    auto store = [&](int h, uint4 u, uint4 w) {
        uint4* dst = h < qh ? qo + h * Dp : reinterpret_cast<uint4*>(ck + (h - qh) * a.c.head_stride);
        if (turns_here) {
            float f[PN];
            Pack<T>::get(u, f);
            if constexpr (INTER) {
#pragma unroll
                for (int e = 0; e < NF; ++e) {
                    const float x = f[2 * e], y = f[2 * e + 1];
                    f[2 * e] = x * cs[e] - y * sn[e];
                    f[2 * e + 1] = x * sn[e] + y * cs[e];
                }
            } else {
                float z[PN];
                Pack<T>::get(w, z);
#pragma unroll
                for (int e = 0; e < NF; ++e) {
                    const float x = f[e], y = z[e];
                    f[e] = x * cs[e] - y * sn[e];
                    z[e] = x * sn[e] + y * cs[e];
                }
                dst[at + Rp / 2] = Pack<T>::put(z);
            }
            u = Pack<T>::put(f);
        }
        dst[at] = u;
    };
#pragma unroll
    for (int e = 0; e < RO_UN; ++e)
        if (g + e * groups < heads) store(g + e * groups, u[e], w[e]);
    // One at a time: in batches the loop took 95 registers instead of 80, and a long prompt 83 us
    // instead of 67.
#pragma unroll 1
    for (int h = g + RO_UN * groups; h < heads; h += groups) {
        load(h, u[0], w[0]);
        store(h, u[0], w[0]);
    }
#pragma unroll 1
    for (int y = tid; y < a.Hkv * Dp; y += RO_THREADS) {
        const int h = y / Dp;
        reinterpret_cast<uint4*>(cv + h * a.c.head_stride)[y - h * Dp] = y == tid ? vv : v[y];
    }
}

template <typename T> void launch(const RotaryArgs& a, unsigned grid, cudaStream_t st) {
    const size_t parents = sizeof(int32_t) * (size_t)a.N;  // N <= 1024 with parents: checked by the caller
    if (a.interleaved) {
        if (a.parent) rotary_kernel<T, true, true><<<grid, RO_THREADS, parents, st>>>(a);
        else rotary_kernel<T, true, false><<<grid, RO_THREADS, 0, st>>>(a);
    } else {
        if (a.parent) rotary_kernel<T, false, true><<<grid, RO_THREADS, parents, st>>>(a);
        else rotary_kernel<T, false, false><<<grid, RO_THREADS, 0, st>>>(a);
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t st) {
    const unsigned grid = (unsigned)a.B * (unsigned)a.N;  // fits: checked by the caller
    if (dtype == TV_BF16) launch<__nv_bfloat16>(a, grid, st);
    else if (dtype == TV_F16) launch<__half>(a, grid, st);
    else launch<float>(a, grid, st);
    return cudaGetLastError();
}

}  // namespace tv
