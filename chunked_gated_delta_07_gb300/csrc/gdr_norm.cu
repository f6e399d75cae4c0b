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
#include "gdr_norm.cuh"

namespace gdr {
namespace {

using namespace norm;

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
    block_partials<kThreads, TPR, NV, VEC>(aw, ab, part, (float *)ring, gi, ri, lane, g, mine, s);
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
    return launch_norm_sum(part, dw, db, (int)n.grid.y, (int64_t)G * D, stream);
}

}  // namespace

cudaError_t launch_norm_sum(const float *part, float *dw, float *db, int nb, int64_t gd, cudaStream_t stream) {
    ProfScope prof(stream, "norm_sum_kernel");
    const cudaError_t err = launch_early(true, norm_sum_kernel, dim3((unsigned)((gd + 31) / 32), 2), 1024, 0, stream,
                                         part, dw, db, nb, gd);
    count_launch();
    return err;
}

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
