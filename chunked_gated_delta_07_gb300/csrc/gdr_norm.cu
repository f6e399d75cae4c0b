// gdr_norm.cu -- layer norm over the last axis, forward and backward, with the
// reduction of the weight's and the bias's gradients.
//
// Rows x_r in R^D; row r uses weight row r % G (G = 1: one weight for all rows; G = H:
// one per head of a [.., H, D] tensor):
//     mu = mean(x),  s = rstd = (mean((x - mu)^2) + eps)^{-1/2},  xh = (x - mu) s
//     y  = xh w + b
//     dx = s (w dy - mean(w dy) - xh mean(w dy xh)),  dw = sum_r dy xh,  db = sum_r dy
// Both passes are bound by HBM: each tensor crosses it once.  A row is held in registers
// by a group of TPR threads (a few lanes of a warp up to a whole block), E elements each,
// so the mean, the squared deviations and the result come from one read; the variance is
// the mean of squared deviations from the mean (no cancellation of large squares).  All
// arithmetic is fp32; inputs and outputs round once.
//
// A block's groups of threads take neighbouring weight rows first, then neighbouring row
// sets, and walk down the rows with the block's stride.  A thread's columns and weight row
// stay the same throughout, so the weight is read once per thread and the backward pass
// sums dw and db in registers; the block adds its groups in a fixed order through shared
// memory and writes one partial sum per (block, column), and a second kernel adds those.
// No atomics: the result is the same on every run.
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

// N consecutive elements of a row as fp32 (N = 1, or a 16-byte piece).
template <typename T, int N> __device__ __forceinline__ void load_n(const T *p, float (&x)[N]) {
    if constexpr (N == 1) {
        x[0] = to_f32(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 v = *(const float4 *)p;
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const uint4 v = *(const uint4 *)p;
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
}
template <typename T, int N> __device__ __forceinline__ void store_n(T *p, const float (&x)[N]) {
    if constexpr (N == 1) {
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

// Sums of NS values over the TPR threads of a row.  Up to a warp: shuffles.  Beyond (the
// block is one row): a shared-memory pass, two buffers taken in turn so that one barrier
// per call is enough.
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
            float x = lane < kW ? red[turn][i][lane] : 0.f;
#pragma unroll
            for (int o = kW / 2; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
            v[i] = __shfl_sync(kFull, x, 0);
        }
        turn ^= 1;
    }
}

// Threads of a block: one row where a row takes more than a warp, else 256.
template <int TPR> constexpr int block_threads() { return TPR > 32 ? TPR : 256; }

template <typename T, int TPR, int NV, int VEC>
__global__ void __launch_bounds__(block_threads<TPR>())
norm_fwd_kernel(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b,
                T *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd, NormShape s) {
    __shared__ float red[2][1][32];
    int turn = 0;
    const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR;
    const int gi = sub % s.gpb, ri = sub / s.gpb;
    const int g = blockIdx.y * s.gpb + gi;
    const bool mine = ri < s.rpb && g < s.G;
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
    // every thread of the block walks the same number of steps (the sums synchronise)
    for (int64_t m0 = (int64_t)blockIdx.x * s.rpb; m0 < s.sets; m0 += (int64_t)gridDim.x * s.rpb) {
        const int64_t m = m0 + ri;
        const bool on = mine && m < s.sets;
        const int64_t row = m * s.G + g, base = row * s.D;
        float xv[NV][VEC], sum[1] = {0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) xv[v][i] = 0.f;
            if (on && c < s.D) load_n<T, VEC>(x + base + c, xv[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[0] += xv[v][i];
        row_sum<TPR, 1>(sum, red, turn);
        const float mu = sum[0] * s.inv_d;
        float sq[1] = {0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = xv[v][i] - mu;
                if ((v * TPR + lane) * VEC < s.D) sq[0] = fmaf(d, d, sq[0]);
            }
        row_sum<TPR, 1>(sq, red, turn);
        const float rs = 1.f / sqrtf(sq[0] * s.inv_d + s.eps);
        if (on) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + lane) * VEC;
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = fmaf((xv[v][i] - mu) * rs, wv[v][i], bv[v][i]);
                if (c < s.D) store_n<T, VEC>(y + base + c, o);
            }
            if (lane == 0) {
                if (mean) mean[row] = mu;
                if (rstd) rstd[row] = rs;
            }
        }
    }
}

// part: [2][gridDim.x][G][D] partial sums of dw, then db (null where neither is wanted).
template <typename T, int TPR, int NV, int VEC>
__global__ void __launch_bounds__(block_threads<TPR>())
norm_bwd_kernel(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
                const float *__restrict__ rstd, const float *__restrict__ w, T *__restrict__ dx,
                float *__restrict__ part, NormShape s) {
    constexpr int kThreads = block_threads<TPR>();
    __shared__ float red[2][2][32];
    __shared__ float comb[TPR > 32 ? 1 : kThreads];
    int turn = 0;
    const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR;
    const int gi = sub % s.gpb, ri = sub / s.gpb;
    const int g = blockIdx.y * s.gpb + gi;
    const bool mine = ri < s.rpb && g < s.G;
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
    for (int64_t m0 = (int64_t)blockIdx.x * s.rpb; m0 < s.sets; m0 += (int64_t)gridDim.x * s.rpb) {
        const int64_t m = m0 + ri;
        const bool on = mine && m < s.sets;
        const int64_t row = m * s.G + g, base = row * s.D;
        float xv[NV][VEC], dv[NV][VEC];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + lane) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) xv[v][i] = dv[v][i] = 0.f;
            if (on && c < s.D) {
                load_n<T, VEC>(x + base + c, xv[v]);
                load_n<T, VEC>(dy + base + c, dv[v]);
            }
        }
        const float mu = on ? mean[row] : 0.f, rs = on ? rstd[row] : 0.f;
        float sum[2] = {0.f, 0.f};   // of w dy, of w dy xh
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool in = on && (v * TPR + lane) * VEC < s.D;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float xh = in ? (xv[v][i] - mu) * rs : 0.f;
                xv[v][i] = xh;
                aw[v][i] = fmaf(dv[v][i], xh, aw[v][i]);
                ab[v][i] += dv[v][i];
                const float wd = dv[v][i] * wv[v][i];
                sum[0] += wd;
                sum[1] = fmaf(wd, xh, sum[1]);
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
                for (int i = 0; i < VEC; ++i) o[i] = rs * (fmaf(dv[v][i], wv[v][i], -c1) - xv[v][i] * c2);
                if (c < s.D) store_n<T, VEC>(dx + base + c, o);
            }
        }
    }
    if (!part) return;
    // the block's partial sums, its row sets added in order
    const int64_t gd = (int64_t)s.G * s.D;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *dst = part + ((int64_t)which * gridDim.x + blockIdx.x) * gd;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int c = (v * TPR + lane) * VEC + i;
                float a = which ? ab[v][i] : aw[v][i];
                if constexpr (TPR <= 32) {
                    if (s.rpb > 1) {
                        __syncthreads();
                        comb[threadIdx.x] = a;
                        __syncthreads();
                        if (ri == 0)
                            for (int r = 1; r < s.rpb; ++r) a += comb[(r * s.gpb + gi) * TPR + lane];
                    }
                }
                if (mine && ri == 0 && c < s.D) dst[(int64_t)g * s.D + c] = a;
            }
    }
}

// out[c] = sum over the nb partial sums of column c, in order; 32 columns x 8 slices of
// the partials per block.
__global__ void __launch_bounds__(256)
norm_sum_kernel(const float *__restrict__ part, float *__restrict__ dw, float *__restrict__ db, int nb,
                int64_t gd) {
    __shared__ float sm[8][33];
    float *out = blockIdx.y ? db : dw;
    if (!out) return;
    const int col = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + col;
    const float *src = part + (int64_t)blockIdx.y * nb * gd + c;
    float a = 0.f;
    if (c < gd)
        for (int i = sl; i < nb; i += 8) a += src[(int64_t)i * gd];
    sm[sl][col] = a;
    __syncthreads();
    if (sl == 0 && c < gd) {
#pragma unroll
        for (int i = 1; i < 8; ++i) a += sm[i][col];
        out[c] = a;
    }
}

// A row's layout over threads: TPR threads with NV pieces of VEC elements each.
struct NormPick {
    int tpr, nv, vec;
};

// The smallest group of threads that holds a row at up to 32 elements a thread: in
// 16-byte pieces where every row can be read that way, else in single elements.
NormPick pick_layout(int D, size_t es, bool pieces) {
    const int vec = pieces ? (int)(16 / es) : 1;
    for (int tpr : {8, 32, 128, 512})
        for (int nv = pieces ? 1 : 32; nv * vec <= 32; nv *= 2)
            if ((int64_t)tpr * nv * vec >= D) return {tpr, nv, vec};
    return {0, 0, 0};
}

// Blocks per SM: enough threads to keep some 40 KB of loads in flight on each SM, few
// enough that the partial sums of the backward pass stay small beside the tensors.
constexpr int kNormThreadsPerSm = 1536;

struct NormGrid {
    dim3 grid;
    int threads;
    NormShape s;
};

NormGrid norm_grid(const NormPick &p, int64_t rows, int G, int D, float eps, int sms) {
    NormGrid o{};
    o.threads = p.tpr > 32 ? p.tpr : 256;
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
    const int64_t most = std::max<int64_t>(1, (int64_t)sms * (kNormThreadsPerSm / o.threads) / by);
    o.grid = dim3((unsigned)std::min(want, most), (unsigned)by);
    return o;
}

// Calls f with the layout as compile-time constants.
template <typename T, typename F> cudaError_t with_layout(const NormPick &p, F &&f) {
    constexpr int V = 16 / sizeof(T);
    using std::integral_constant;
#define GDR_NORM_CASE(TPR_, NV_, VEC_)                                                             \
    if (p.tpr == TPR_ && p.nv == NV_ && p.vec == VEC_)                                             \
        return f(integral_constant<int, TPR_>{}, integral_constant<int, NV_>{}, integral_constant<int, VEC_>{});
    GDR_NORM_CASE(8, 1, V)
    GDR_NORM_CASE(8, 2, V)
    GDR_NORM_CASE(8, 4, V)
    GDR_NORM_CASE(32, 2, V)
    GDR_NORM_CASE(32, 4, V)
    GDR_NORM_CASE(128, 2, V)
    GDR_NORM_CASE(128, 4, V)
    GDR_NORM_CASE(512, 2, V)
    GDR_NORM_CASE(512, 4, V)
    if constexpr (sizeof(T) == 4) {
        GDR_NORM_CASE(8, 8, V)
        GDR_NORM_CASE(32, 8, V)
        GDR_NORM_CASE(128, 8, V)
        GDR_NORM_CASE(512, 8, V)
    }
    GDR_NORM_CASE(8, 32, 1)
    GDR_NORM_CASE(32, 32, 1)
    GDR_NORM_CASE(128, 32, 1)
    GDR_NORM_CASE(512, 32, 1)
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
    const NormGrid n = norm_grid(p, rows, G, D, eps, sms);
    return with_layout<T>(p, [&](auto tpr, auto nv, auto vec) {
        ProfScope prof(stream, "norm_fwd_kernel");
        norm_fwd_kernel<T, tpr(), nv(), vec()><<<n.grid, n.threads, 0, stream>>>(
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
    const NormGrid n = norm_grid(p, rows, G, D, 0.f, sms);
    float *part = dw || db ? scratch : nullptr;
    const cudaError_t err = with_layout<T>(p, [&](auto tpr, auto nv, auto vec) {
        ProfScope prof(stream, "norm_bwd_kernel");
        norm_bwd_kernel<T, tpr(), nv(), vec()><<<n.grid, n.threads, 0, stream>>>(
            (const T *)dy, (const T *)x, mean, rstd, w, (T *)dx, part, n.s);
        count_launch();
        return cudaGetLastError();
    });
    if (err != cudaSuccess || !part) return err;
    const int64_t gd = (int64_t)G * D;
    ProfScope prof(stream, "norm_sum_kernel");
    norm_sum_kernel<<<dim3((unsigned)((gd + 31) / 32), 2), 256, 0, stream>>>(part, dw, db, (int)n.grid.x, gd);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_scratch_bytes(int64_t rows, int G, int D, gdr_dtype_t dtype, int sms) {
    const size_t es = dtype == GDR_BF16 ? 2 : 4;
    size_t need = 0;   // whichever layout the pointers' alignment allows
    for (bool pieces : {true, false})
        need = std::max(need, sizeof(float) * 2 * norm_grid(pick_layout(D, es, pieces), rows, G, D, 0.f, sms).grid.x *
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
