// gdr_norm.cu -- layer norm over the last axis, forward and backward, with the
// reduction of the weight's and the bias's gradients.
//
// Rows x_r in R^D; row r uses weight row r % G (G = 1: one weight for all rows; G = H:
// one per head of a [.., H, D] tensor):
//     mu = mean(x),  s = rstd = (mean((x - mu)^2) + eps)^{-1/2},  xh = (x - mu) s
//     y  = xh w + b
//     dx = s (w dy - mean(w dy) - xh mean(w dy xh)),  dw = sum_r dy xh,  db = sum_r dy
// Both passes are bound by HBM: each tensor crosses it once.  A row is held in registers by
// a group of TPR threads (a few lanes of a warp up to a whole block), 8 elements each (16 in
// the widest rows), so the mean, the squared deviations and the result come from one read;
// the variance is the mean of squared deviations from the mean (no cancellation of large
// squares).  The loads of the next rows are on their way while a row is computed.  All
// arithmetic is fp32; inputs and outputs round once.
//
// A block's groups of threads take neighbouring weight rows first, then neighbouring row
// sets, and walk down the rows with the block's stride.  A thread's columns and weight row
// stay the same throughout, so the weight is read once per thread and the backward pass
// sums dw and db in registers; the block adds its groups in a fixed order through shared
// memory and writes one partial sum per (block, column), and a second kernel adds those.
// No atomics: the result is the same on every run.
//
// Measured (bf16): 524288 rows x 128 with 16 weight rows forward 47.6 us, 5.7 TB/s, 84% of a
// copy's; backward 71.5 us, 5.7 TB/s.  8191 rows x 2048 backward 29.0 us, 3.5 TB/s: with 14 pairs
// of rows to a block, the first loads, the last stores and the sum of 304 partials weigh as much
// as the rows between them.  16 elements a thread, which halves the threads of a row's exchanges,
// gave 48.4, 167 and 65 us.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "gdr_internal.cuh"

namespace gdr {
namespace {

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
template <int NV, int TENSORS> constexpr int ring_depth() {
    constexpr int fit = kRingBytesPerSm / (kThreadsPerSm * 16 * NV * TENSORS);
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

template <typename T, int TPR, int NV, int VEC>
__global__ void __launch_bounds__(fwd_threads<TPR>())
norm_fwd_kernel(const T *x, const float *__restrict__ w, const float *__restrict__ b, T *y,
                float *__restrict__ mean, float *__restrict__ rstd, NormShape s) {
    __shared__ float red[2][1][32];
    int turn = 0;
    const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR;
    const int gi = sub % s.gpb, ri = sub / s.gpb;
    const int g = blockIdx.x * s.gpb + gi;
    const bool mine = ri < s.rpb && g < s.G;
    constexpr int kDepth = VEC > 1 ? ring_depth<NV, 1>() : 2;
    extern __shared__ uint4 ring[];
    const int64_t step = (int64_t)gridDim.y * s.rpb, row_step = step * s.G;
    int64_t m = (int64_t)blockIdx.y * s.rpb + ri, row = m * s.G + g;
    RowStream<T, fwd_threads<TPR>(), TPR, NV, VEC> xs{};
    xs.p = x + row * s.D + lane * VEC;
    xs.step = row_step * s.D;
    xs.ring = ring + threadIdx.x;
    xs.p0 = x;
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) {
        xs.ask(i, lane, s.D, mine && m + i * step < s.sets);
        copies_commit();
    }
    float wv[NV][VEC], bv[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (v * TPR + lane) * VEC + i;
            const bool in = mine && c < s.D;
            wv[v][i] = in && w ? w[(int64_t)g * s.D + c] : 1.f;
            bv[v][i] = in && b ? b[(int64_t)g * s.D + c] : 0.f;
        }
    // every thread of the block takes the same number of steps (the sums synchronise)
    int slot = 0;
    for (int64_t m0 = m - ri; m0 < s.sets; m0 += step, m += step, row += row_step) {
        const bool on = mine && m < s.sets;
        // the slot asked for is the one read a step ago
        xs.ask(slot == 0 ? kDepth - 1 : slot - 1, lane, s.D, mine && m + (kDepth - 1) * step < s.sets);
        copies_commit();
        copies_wait<kDepth - 1>();
        typename Piece<T, VEC>::type raw[NV];
        xs.read(slot, raw);
        slot = slot == kDepth - 1 ? 0 : slot + 1;
        float xv[NV][VEC], sum[1] = {0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            widen<T, VEC>(raw[v], xv[v]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[0] += xv[v][i];
        }
        row_sum<TPR, 1>(sum, red, turn);
        const float mu = sum[0] * s.inv_d;
        float sq[1] = {0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                xv[v][i] -= mu;
                if ((v * TPR + lane) * VEC < s.D) sq[0] = fmaf(xv[v][i], xv[v][i], sq[0]);
            }
        row_sum<TPR, 1>(sq, red, turn);
        const float rs = rsqrtf(sq[0] * s.inv_d + s.eps);   // within 2^-22 of its value
        if (on) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + lane) * VEC;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = fmaf(xv[v][i] * rs, wv[v][i], bv[v][i]);
                if (c < s.D) store_n<T, VEC>(y + row * s.D + c, o);
            }
            if (lane == 0) {
                if (mean) mean[row] = mu;
                if (rstd) rstd[row] = rs;
            }
        }
    }
}

// part: [2][gridDim.y][G][D] partial sums of dw, then db (null where neither is wanted).
// Rows in single elements get twice the registers, one block of 512 threads at a time: with two,
// 8 elements' sums, weights and addresses do not fit (the kernel alone, with dy = x: 65537 rows x
// 999 bf16 208 us, with one 110; 200000 x 125 137 and 66).  Rows in 16-byte pieces fit.
template <typename T, int TPR, int NV, int VEC>
__global__ void __launch_bounds__(bwd_threads<TPR>(), VEC > 1 ? kThreadsPerSm / bwd_threads<TPR>() : 1)
norm_bwd_kernel(const T *dy, const T *x, const float *__restrict__ mean, const float *__restrict__ rstd,
                const float *__restrict__ w, T *dx, float *__restrict__ part, NormShape s) {
    constexpr int kThreads = bwd_threads<TPR>();
    __shared__ float red[2][2][32];
    let_next_start();
    int turn = 0;
    const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR;
    const int gi = sub % s.gpb, ri = sub / s.gpb;
    const int g = blockIdx.x * s.gpb + gi;
    const bool mine = ri < s.rpb && g < s.G;
    const int64_t step = (int64_t)gridDim.y * s.rpb, row_step = step * s.G;
    int64_t m = (int64_t)blockIdx.y * s.rpb + ri, row = m * s.G + g;
    constexpr int kDepth = VEC > 1 ? ring_depth<NV, 2>() : 2;
    extern __shared__ uint4 ring[];
    RowStream<T, kThreads, TPR, NV, VEC> xs{}, ds{};
    xs.p = x + row * s.D + lane * VEC;
    ds.p = dy + row * s.D + lane * VEC;
    xs.step = ds.step = row_step * s.D;
    xs.ring = ring + threadIdx.x;
    ds.ring = xs.ring + kDepth * NV * kThreads;
    xs.p0 = x;
    ds.p0 = dy;
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) {
        const bool on = mine && m + i * step < s.sets;
        xs.ask(i, lane, s.D, on);
        ds.ask(i, lane, s.D, on);
        copies_commit();
    }
    float mu = mine && m < s.sets ? mean[row] : 0.f, rs = mine && m < s.sets ? rstd[row] : 0.f;
    float wv[NV][VEC], aw[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (v * TPR + lane) * VEC + i;
            wv[v][i] = mine && c < s.D && w ? w[(int64_t)g * s.D + c] : 1.f;
            aw[v][i] = 0.f;
            ab[v][i] = 0.f;
        }
    int slot = 0;
    for (int64_t m0 = m - ri; m0 < s.sets; m0 += step, m += step, row += row_step) {
        const bool on = mine && m < s.sets;
        const bool ask = mine && m + (kDepth - 1) * step < s.sets;
        const int back = slot == 0 ? kDepth - 1 : slot - 1;   // the slot read a step ago
        xs.ask(back, lane, s.D, ask);
        ds.ask(back, lane, s.D, ask);
        copies_commit();
        const bool more = mine && m + step < s.sets;
        const float mu1 = more ? mean[row + row_step] : 0.f, rs1 = more ? rstd[row + row_step] : 0.f;
        copies_wait<kDepth - 1>();
        typename Piece<T, VEC>::type rx[NV], rd[NV];
        xs.read(slot, rx);
        ds.read(slot, rd);
        slot = slot == kDepth - 1 ? 0 : slot + 1;
        float xv[NV][VEC], dv[NV][VEC], sum[2] = {0.f, 0.f};   // of w dy, of w dy xh
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool in = on && (v * TPR + lane) * VEC < s.D;
            widen<T, VEC>(rx[v], xv[v]);
            widen<T, VEC>(rd[v], dv[v]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float xh = in ? (xv[v][i] - mu) * rs : 0.f;
                xv[v][i] = xh;
                aw[v][i] = fmaf(dv[v][i], xh, aw[v][i]);
                ab[v][i] += dv[v][i];
                dv[v][i] *= wv[v][i];
                sum[0] += dv[v][i];
                sum[1] = fmaf(dv[v][i], xh, sum[1]);
            }
        }
        row_sum<TPR, 2>(sum, red, turn);
        const float c1 = sum[0] * s.inv_d, c2 = sum[1] * s.inv_d;
        if (on) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + lane) * VEC;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = rs * (dv[v][i] - c1 - xv[v][i] * c2);
                if (c < s.D) store_n<T, VEC>(dx + row * s.D + c, o);
            }
        }
        mu = mu1;
        rs = rs1;
    }
    // no copy of this thread's may still be on its way into the ring: those asked for past the
    // last row fill it with zeros, and its memory is taken for the groups' sums below
    copies_wait<0>();
    if (!part) return;
    // the block's partial sums, its row sets added in order through shared memory
    const int64_t gd = (int64_t)s.G * s.D;
    float *comb = (float *)ring;   // [NV * VEC][threads]
    const int first = gi * TPR + lane;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float(&a)[NV][VEC] = which ? ab : aw;
        if (TPR < kThreads && s.rpb > 1) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NV * VEC; ++k) comb[k * kThreads + threadIdx.x] = a[k / VEC][k % VEC];
            __syncthreads();
            if (mine && ri == 0)
                for (int r = 1; r < s.rpb; ++r)
#pragma unroll
                    for (int k = 0; k < NV * VEC; ++k)
                        a[k / VEC][k % VEC] += comb[k * kThreads + r * s.gpb * TPR + first];
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

// out[c] = sum over the nb partial sums of column c, in a fixed order: 32 columns x 32
// slices of the partials per block.  Bound by its start and the loads' latency: 6 us for
// 5 MB of partials out of the L2, 2 to 3 of them behind the end of the pass (launched early).
__global__ void __launch_bounds__(1024)
norm_sum_kernel(const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ db, int nb,
                int64_t gd) {
    __shared__ float sm[32][33];
    after_previous();
    float *out = blockIdx.y ? db : dw;
    if (!out) return;
    const int col = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + col;
    const float *src = part + (int64_t)blockIdx.y * nb * gd + c;
    float a = 0.f;
    if (c < gd)
#pragma unroll 8
        for (int i = sl; i < nb; i += 32) a += src[(int64_t)i * gd];
    sm[sl][col] = a;
    __syncthreads();
    // warp sl adds the slices of column sl
    a = sm[col][sl];
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
    if (col == 0 && (int64_t)blockIdx.x * 32 + sl < gd) out[(int64_t)blockIdx.x * 32 + sl] = a;
}

// A row's layout over threads: TPR threads with NV pieces of VEC elements each.
struct NormPick {
    int tpr, nv, vec;
};

// The smallest group of threads that holds a row at 8 elements a thread (16 beyond 8192
// columns): in 16-byte pieces where every row can be read that way, else in single elements, of
// which 512 threads take 16 (the kernel alone: 20000 rows x 6001 fp32 backward, dy = x, 307 us, 1024
// threads with 8 370; 4097 bf16 forward 138 and 170).
NormPick pick_layout(int D, size_t es, bool pieces) {
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

NormGrid norm_grid(const NormPick &p, int64_t rows, int G, int D, float eps, int sms, int least) {
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
    const int64_t most = std::max<int64_t>(1, (int64_t)sms * (kThreadsPerSm / o.threads) / by);
    o.grid = dim3((unsigned)by, (unsigned)std::min(want, most));
    return o;
}

// Calls f with the layout as compile-time constants.
template <typename T, typename F> cudaError_t with_layout(const NormPick &p, F &&f) {
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
    GDR_NORM_CASE(1024, 16, 1)
#undef GDR_NORM_CASE
    return cudaErrorInvalidValue;
}

bool in_pieces(int D, size_t es, std::initializer_list<const void *> ptrs) {
    if (D % (16 / es)) return false;
    for (const void *p : ptrs)
        if ((uintptr_t)p % 16) return false;
    return true;
}

template <typename T>
cudaError_t fwd_t(const void *x, const float *w, const float *b, void *y, float *mean, float *rstd,
                  int64_t rows, int G, int D, float eps, int sms, cudaStream_t stream) {
    const NormPick p = pick_layout(D, sizeof(T), in_pieces(D, sizeof(T), {x, y}));
    const NormGrid n = norm_grid(p, rows, G, D, eps, sms, 256);
    return with_layout<T>(p, [&](auto tpr, auto nv, auto vec) {
        auto kern = norm_fwd_kernel<T, tpr(), nv(), vec()>;
        const int smem = vec() > 1 ? ring_depth<nv(), 1>() * n.threads * 16 * nv() : 0;
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
        ProfScope prof(stream, "norm_fwd_kernel");
        kern<<<n.grid, n.threads, smem, stream>>>(
            (const T *)x, w, b, (T *)y, mean, rstd, n.s);
        count_launch();
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t bwd_t(const void *dy, const void *x, const float *mean, const float *rstd, const float *w,
                  void *dx, float *dw, float *db, int64_t rows, int G, int D, int sms,
                  float *scratch, cudaStream_t stream) {
    const NormPick p = pick_layout(D, sizeof(T), in_pieces(D, sizeof(T), {dy, x, dx}));
    const NormGrid n = norm_grid(p, rows, G, D, 0.f, sms, 512);
    float *part = dw || db ? scratch : nullptr;
    const cudaError_t err = with_layout<T>(p, [&](auto tpr, auto nv, auto vec) {
        auto kern = norm_bwd_kernel<T, tpr(), nv(), vec()>;
        const int smem = std::max(vec() > 1 ? ring_depth<nv(), 2>() * n.threads * 32 * nv() : 0,
                                  n.threads * 4 * nv() * vec());
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
        ProfScope prof(stream, "norm_bwd_kernel");
        kern<<<n.grid, n.threads, smem, stream>>>(
            (const T *)dy, (const T *)x, mean, rstd, w, (T *)dx, part, n.s);
        count_launch();
        return cudaGetLastError();
    });
    if (err != cudaSuccess || !part) return err;
    const int64_t gd = (int64_t)G * D;
    ProfScope prof(stream, "norm_sum_kernel");
    const cudaError_t sum = launch_early(true, norm_sum_kernel, dim3((unsigned)((gd + 31) / 32), 2), 1024, 0, stream,
                                         (const float *)part, dw, db, (int)n.grid.y, gd);
    count_launch();
    return sum;
}

}  // namespace

size_t norm_bwd_scratch_bytes(int64_t rows, int G, int D, gdr_dtype_t dtype, int sms) {
    const size_t es = dtype == GDR_BF16 ? 2 : 4;
    size_t need = 0;   // whichever layout the pointers' alignment allows
    for (bool pieces : {true, false})
        need = std::max(need, sizeof(float) * 2 * norm_grid(pick_layout(D, es, pieces), rows, G, D, 0.f, sms, 512).grid.y *
                                  (size_t)G * D);
    return need;
}

cudaError_t launch_norm_fwd(const void *x, const float *w, const float *b, void *y, float *mean, float *rstd,
                            int64_t rows, int G, int D, float eps, gdr_dtype_t dtype, int sms,
                            cudaStream_t stream) {
    return dtype == GDR_BF16 ? fwd_t<__nv_bfloat16>(x, w, b, y, mean, rstd, rows, G, D, eps, sms, stream)
                             : fwd_t<float>(x, w, b, y, mean, rstd, rows, G, D, eps, sms, stream);
}

cudaError_t launch_norm_bwd(const void *dy, const void *x, const float *mean, const float *rstd, const float *w,
                            void *dx, float *dw, float *db, int64_t rows, int G, int D, gdr_dtype_t dtype,
                            int sms, float *scratch, cudaStream_t stream) {
    return dtype == GDR_BF16
               ? bwd_t<__nv_bfloat16>(dy, x, mean, rstd, w, dx, dw, db, rows, G, D, sms, scratch, stream)
               : bwd_t<float>(dy, x, mean, rstd, w, dx, dw, db, rows, G, D, sms, scratch, stream);
}

}  // namespace gdr
