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
// One CTA per node.  While the first R/2 threads form the angles, every
// thread's first loads are already under way.  Bound: HBM (each row is read
// once and written once).
#include "kernels.h"
#include "tv_common.cuh"

namespace tv {
namespace {

constexpr int RO_THREADS = 256;

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

// Depth of node j (steps to the root), or -1 when its path is malformed.
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

template <typename T>
__global__ void __launch_bounds__(RO_THREADS) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    constexpr int PN = Pack<T>::N;
    __shared__ float s_cos[128], s_sin[128];
    __shared__ long long s_off;
    __shared__ int s_bad, s_depth;
    const int tid = threadIdx.x, b = blockIdx.x / a.N, j = blockIdx.x - b * a.N;
    bool bad_count;
    const int n = seq_nodes(a.counts, b, a.N, bad_count);
    if (j >= n) return;
    const int L = a.prefix_lens[b];
    if (tid == 0) {
        int bad = 0, depth = j;
        long long off = -1;
        if (bad_count || L < 0 || (long long)L + n > (long long)a.c.max_blocks * a.c.block_size) {
            bad = TV_ERR_INVALID_ARG;
        } else {
            const int t = L + j, blk = t / a.c.block_size;
            const int id = a.c.table[(size_t)b * a.c.max_blocks + blk];
            if (id < 0 || id >= a.c.num_blocks) bad = TV_ERR_BLOCK_TABLE;
            else off = (long long)id * a.c.block_stride + (long long)(t - blk * a.c.block_size) * a.c.token_stride;
            if (a.parent) {
                depth = node_depth(a.parent + (size_t)b * a.N, j);
                if (depth < 0) bad = TV_ERR_TREE;
            }
        }
        s_bad = bad;
        s_off = off;
        s_depth = depth;
        if (bad) report(a.status, bad);
    }
    __syncthreads();
    const int bad = s_bad;
    if (!bad) {
        for (int i = tid; i < a.rot / 2; i += RO_THREADS) {
            const int ax = a.axis_of_pair[i];
            double pos;
            if (a.positions) pos = (double)a.positions[((size_t)ax * a.B + b) * a.N + j];
            else pos = (double)(a.position_base ? a.position_base[b] : L) + (double)s_depth;
            const double turns = pos * (double)a.inv_freq[i] * 0.15915494309189533577;
            float sn, cs;
            sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
            s_cos[i] = cs;
            s_sin[i] = sn;
        }
    }
    __syncthreads();
    const int Dp = a.D / PN, Rp = a.rot / PN;    // 16-byte pieces of a row; rotated pieces
    const size_t node = (size_t)b * a.N + j;
    const uint4* q = a.q ? reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + node * a.q_stride) : nullptr;
    uint4* qo = reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + node * (size_t)a.Hq * a.D);
    const uint4* k = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + node * a.k_stride);
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + node * a.v_stride);
    if (bad) {
        if (q) {
            float nanv[PN];
#pragma unroll
            for (int e = 0; e < PN; ++e) nanv[e] = __int_as_float(0x7fc00000);
            for (int i = tid; i < a.Hq * Dp; i += RO_THREADS) qo[i] = Pack<T>::put(nanv);
        }
    } else {
        char* ck = static_cast<char*>(a.cache_k) + s_off;
        char* cv = static_cast<char*>(a.cache_v) + s_off;
        const int heads = (q ? a.Hq : 0) + a.Hkv;
        // split halves: a unit is the pieces i and i + R/2; neighbouring pairs: one piece
        const int units = a.interleaved ? Dp : Dp - Rp / 2;
        for (int x = tid; x < heads * units; x += RO_THREADS) {
            const int hh = x / units, i = x - hh * units;
            const bool isq = q && hh < a.Hq;
            const int h = isq || !q ? hh : hh - a.Hq;
            const uint4* src = (isq ? q : k) + (size_t)h * Dp;
            uint4* dst = isq ? qo + (size_t)h * Dp : reinterpret_cast<uint4*>(ck + h * a.c.head_stride);
            float f[PN], g[PN], r[PN];
            if (a.interleaved) {
                const uint4 u = src[i];
                if (i >= Rp) { dst[i] = u; continue; }
                Pack<T>::get(u, f);
#pragma unroll
                for (int e = 0; e < PN; e += 2) {
                    const float cs = s_cos[(i * PN + e) / 2], sn = s_sin[(i * PN + e) / 2];
                    r[e] = f[e] * cs - f[e + 1] * sn;
                    r[e + 1] = f[e] * sn + f[e + 1] * cs;
                }
                dst[i] = Pack<T>::put(r);
            } else if (i < Rp / 2) {
                const uint4 u = src[i], w = src[i + Rp / 2];
                Pack<T>::get(u, f);
                Pack<T>::get(w, g);
                float r2[PN];
#pragma unroll
                for (int e = 0; e < PN; ++e) {
                    const float cs = s_cos[i * PN + e], sn = s_sin[i * PN + e];
                    r[e] = f[e] * cs - g[e] * sn;
                    r2[e] = f[e] * sn + g[e] * cs;
                }
                dst[i] = Pack<T>::put(r);
                dst[i + Rp / 2] = Pack<T>::put(r2);
            } else {
                dst[i + Rp / 2] = src[i + Rp / 2];  // past the rotated part
            }
        }
        for (int x = tid; x < a.Hkv * Dp; x += RO_THREADS) {
            const int h = x / Dp, i = x - h * Dp;
            reinterpret_cast<uint4*>(cv + h * a.c.head_stride)[i] = v[(size_t)h * Dp + i];
        }
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t st) {
    const unsigned grid = (unsigned)a.B * (unsigned)a.N;  // fits: checked by the caller
    if (dtype == TV_BF16) rotary_kernel<__nv_bfloat16><<<grid, RO_THREADS, 0, st>>>(a);
    else if (dtype == TV_F16) rotary_kernel<__half><<<grid, RO_THREADS, 0, st>>>(a);
    else rotary_kernel<float><<<grid, RO_THREADS, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace tv
