// gdr_norm.cuh -- what the kernels that norm rows share: rows held in registers by groups of
// threads, streamed through a ring in shared memory, sums over a row's threads, and the choice
// of the layout.
#pragma once

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "gdr_internal.cuh"

namespace gdr {
namespace norm {

constexpr unsigned kFull = 0xffffffffu;

struct NormShape {
    int64_t sets;   // rows / G
    int G, D;
    float eps, inv_d;
    int gpb, rpb;   // weight rows and row sets of a block's thread groups
};

// VEC consecutive elements of a row as they are in memory: one element, or 16 bytes.
template <typename T, int VEC> struct Piece {
    using type = uint4;
};
template <typename T> struct Piece<T, 1> {
    using type = T;
};

template <typename T, int VEC>
__device__ __forceinline__ void widen(const typename Piece<T, VEC>::type &v, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = to_f32(v);
    } else {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(u[i]);
            } else {
                x[2 * i] = __uint_as_float(u[i] << 16);
                x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        }
    }
}
template <typename T, int VEC> __device__ __forceinline__ void store_n(T *p, const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        *p = from_f32<T>(x[0]);
    } else if constexpr (sizeof(T) == 4) {
        *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *(const uint32_t *)&h;
        }
        *(uint4 *)p = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// Threads of a block: at least 256 (several rows), up to a row's; at least 512 in the
// backward pass, whose blocks each write a partial sum of the weights' gradients.
template <int TPR> constexpr int fwd_threads() { return TPR > 256 ? TPR : 256; }
template <int TPR> constexpr int bwd_threads() { return TPR > 512 ? TPR : 512; }
// Of either pass on an SM, as its registers allow (1536 in the forward pass: 60 us for the first
// call above against 48).
constexpr int kThreadsPerSm = 1024;

// Rows under way per thread: loads of 16-byte pieces go through a ring in shared memory
// (asynchronous copies, each thread reading back its own: no barrier), 4 rows deep where the
// SM's blocks have room for it; single elements are loaded one row ahead in registers.
constexpr int kRingBytesPerSm = 200 * 1024;
template <int NV, int TENSORS, int PER_SM = kThreadsPerSm> constexpr int ring_depth() {
    constexpr int fit = kRingBytesPerSm / (PER_SM * 16 * NV * TENSORS);
    return fit > 4 ? 4 : fit;
}

// The rows of one tensor as a thread takes them, one call of next() per step; `ahead` rows
// have been asked for when a row is read.
template <typename T, int THREADS, int TPR, int NV, int VEC> struct RowStream {
    const T *p;        // the thread's first column in the next row to ask for
    int64_t step;      // elements from row to row of the thread
    uint4 *ring;       // [depth][NV][THREADS], at the thread
    __device__ __forceinline__ void ask(int slot, int lane, int D, bool on) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + lane) * VEC;
            const unsigned dst = (unsigned)__cvta_generic_to_shared(ring + (slot * NV + i) * THREADS);
            const int bytes = on && c < D ? 16 : 0;   // the rest of the 16 is filled with zeros
            const T *src = bytes ? p + i * TPR * VEC : p0;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
        }
        p += step;
    }
    const T *p0;       // any valid address of the tensor
    __device__ __forceinline__ void read(int slot, uint4 (&v)[NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = ring[(slot * NV + i) * THREADS];
    }
};
template <typename T, int THREADS, int TPR, int NV> struct RowStream<T, THREADS, TPR, NV, 1> {
    const T *p;
    int64_t step;
    uint4 *ring;       // not used
    T next[NV], cur[NV];
    __device__ __forceinline__ void ask(int, int lane, int D, bool on) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            cur[i] = next[i];
            next[i] = on && i * TPR + lane < D ? p[i * TPR] : from_f32<T>(0.f);
        }
        p += step;
    }
    const T *p0;
    __device__ __forceinline__ void read(int, T (&v)[NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = cur[i];
    }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sums of NS values over the TPR threads of a row.  Up to a warp: shuffles.  Beyond: a
// shared-memory pass over the row's warps, two buffers taken in turn so that one barrier per
// call is enough (every thread of the block calls).
template <int TPR, int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], float (*red)[NS][32], int &turn) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < NS; ++i) v[i] += __shfl_xor_sync(kFull, v[i], o);
    if constexpr (TPR > 32) {
        constexpr int kW = TPR / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) red[turn][i][warp] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float x = lane < kW ? red[turn][i][warp / kW * kW + lane] : 0.f;
#pragma unroll
            for (int o = kW / 2; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
            v[i] = __shfl_sync(kFull, x, 0);
        }
        turn ^= 1;
    }
}

// A block's partial sums aw and ab of the weights' gradients, its row sets added in order through
// shared memory (comb: [NV * VEC][THREADS] floats), into part [2][gridDim.y][G][D]; every thread of
// the block calls, with no copy into that memory under way.
template <int THREADS, int TPR, int NV, int VEC>
__device__ __forceinline__ void block_partials(float (&aw)[NV][VEC], float (&ab)[NV][VEC], float *__restrict__ part,
                                               float *comb, int gi, int ri, int lane, int g, bool mine,
                                               const NormShape &s) {
    const int64_t gd = (int64_t)s.G * s.D;
    const int first = gi * TPR + lane;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float(&a)[NV][VEC] = which ? ab : aw;
        if (TPR < THREADS && s.rpb > 1) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NV * VEC; ++k) comb[k * THREADS + threadIdx.x] = a[k / VEC][k % VEC];
            __syncthreads();
            if (mine && ri == 0)
                for (int r = 1; r < s.rpb; ++r)
#pragma unroll
                    for (int k = 0; k < NV * VEC; ++k)
                        a[k / VEC][k % VEC] += comb[k * THREADS + r * s.gpb * TPR + first];
        }
        if (!mine || ri != 0) continue;
        float *dst = part + ((int64_t)which * gridDim.y + blockIdx.y) * gd + (int64_t)g * s.D;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * VEC;
            if (c >= s.D) continue;
            if constexpr (VEC % 4 == 0) {   // D is a multiple of VEC
#pragma unroll
                for (int i = 0; i < VEC; i += 4)
                    *(float4 *)(dst + c + i) = make_float4(a[v][i], a[v][i + 1], a[v][i + 2], a[v][i + 3]);
            } else {
                dst[c] = a[v][0];
            }
        }
    }
}

// A row's layout over threads: TPR threads with NV pieces of VEC elements each.
struct NormPick {
    int tpr, nv, vec;
};

// The smallest group of threads that holds a row at 8 elements a thread (16 beyond 8192
// columns): in 16-byte pieces where every row can be read that way, else in single elements, of
// which 512 threads take 16 (the kernel alone: 20000 rows x 6001 fp32 backward, dy = x, 307 us, 1024
// threads with 8 370; 4097 bf16 forward 138 and 170).
inline NormPick pick_layout(int D, size_t es, bool pieces) {
    const int vec = pieces ? (int)(16 / es) : 1, nv = 8 / vec;
    for (int tpr = 8; tpr <= 1024; tpr *= pieces ? 2 : 4)
        if (tpr * 8 >= D) return {tpr, nv, vec};
    return {!pieces && D <= 8192 ? 512 : 1024, 2 * nv, vec};
}

struct NormGrid {
    dim3 grid;   // groups of weight rows (up to 2^20) x blocks along the row sets
    int threads;
    NormShape s;
};

inline NormGrid norm_grid(const NormPick &p, int64_t rows, int G, int D, float eps, int sms, int least,
                          int per_sm = kThreadsPerSm) {
    NormGrid o{};
    o.threads = std::max(p.tpr, least);
    const int subs = o.threads / p.tpr;
    o.s.sets = rows / G;
    o.s.G = G;
    o.s.D = D;
    o.s.eps = eps;
    o.s.inv_d = 1.f / (float)D;
    o.s.gpb = std::min(G, subs);
    o.s.rpb = subs / o.s.gpb;
    const int64_t by = (G + o.s.gpb - 1) / o.s.gpb;
    const int64_t want = (o.s.sets + o.s.rpb - 1) / o.s.rpb;
    const int64_t most = std::max<int64_t>(1, (int64_t)sms * std::max(1, per_sm / o.threads) / by);
    o.grid = dim3((unsigned)by, (unsigned)std::min(want, most));
    return o;
}

// Calls f with the layout as compile-time constants (WIDE: single elements also 8 to each of 16, 64, 256
// or 1024 threads).
template <typename T, bool WIDE = false, typename F> cudaError_t with_layout(const NormPick &p, F &&f) {
    constexpr int V = 16 / sizeof(T);
    using std::integral_constant;
#define GDR_NORM_CASE(TPR_, NV_, VEC_)                                                             \
    if (p.tpr == TPR_ && p.nv == NV_ && p.vec == VEC_)                                             \
        return f(integral_constant<int, TPR_>{}, integral_constant<int, NV_>{}, integral_constant<int, VEC_>{});
    constexpr int N = 8 / V;
    GDR_NORM_CASE(8, N, V)
    GDR_NORM_CASE(16, N, V)
    GDR_NORM_CASE(32, N, V)
    GDR_NORM_CASE(64, N, V)
    GDR_NORM_CASE(128, N, V)
    GDR_NORM_CASE(256, N, V)
    GDR_NORM_CASE(512, N, V)
    GDR_NORM_CASE(1024, N, V)
    GDR_NORM_CASE(1024, 2 * N, V)
    GDR_NORM_CASE(8, 8, 1)
    GDR_NORM_CASE(32, 8, 1)
    GDR_NORM_CASE(128, 8, 1)
    GDR_NORM_CASE(512, 8, 1)
    GDR_NORM_CASE(512, 16, 1)
    if constexpr (WIDE) {
        GDR_NORM_CASE(16, 8, 1)
        GDR_NORM_CASE(64, 8, 1)
        GDR_NORM_CASE(256, 8, 1)
        GDR_NORM_CASE(1024, 8, 1)
    }
    GDR_NORM_CASE(1024, 16, 1)
#undef GDR_NORM_CASE
    return cudaErrorInvalidValue;
}

inline bool in_pieces(int D, size_t es, std::initializer_list<const void *> ptrs) {
    if (D % (16 / es)) return false;
    for (const void *p : ptrs)
        if ((uintptr_t)p % 16) return false;
    return true;
}

}  // namespace norm

// dw, db [gd] = the sums over the nb partial sums of each column (part [2][nb][gd]), in a fixed
// order; dw or db may be null.
cudaError_t launch_norm_sum(const float *part, float *dw, float *db, int nb, int64_t gd, cudaStream_t stream);

}  // namespace gdr
