// gdr_block_norm_fwd.cu -- the forward passes of the norms around a block (gdr_block_norm.cuh).
//
// Bound by HBM: each tensor crosses it once.  As in the layer norm, a row is held in the
// registers of a group of threads, 8 elements each, and the next rows of every input are on
// their way through a ring in shared memory; the variance is the mean of squared deviations.
// Measured (bf16): add_norm 32768 x 2048 95 us, 5.6 TB/s, 85% of a copy's rate; norm_gate 524288 x
// 128 with 16 weight rows 65 to 68 us, 6.0 TB/s, 89 to 93% (28 instructions an element, 78% of the
// issue slots).
// add_norm norms the sum as it is stored, rounded to the tensors' type, so that the backward
// pass, which reads that sum, differentiates what was computed.
#include "gdr_block_norm.cuh"

namespace gdr {
namespace {

using namespace norm;

// Mean (0 for rms) and reciprocal deviation of a row held in xv, which is centred in place.
template <typename P, int TPR, int NV, int VEC, int KP, typename V>
__device__ __forceinline__ void row_stats(V (&xv)[NV][KP], int lane, const NormShape &s, bool rms, float (*red)[1][32],
                                          int &turn, float &mu, float &rs) {
    mu = 0.f;
    if (!rms) {
        V acc = P::of(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < KP; ++i) acc = add2(acc, xv[v][i]);
        float sum[1] = {P::sum(acc)};
        row_sum<TPR, 1>(sum, red, turn);
        mu = sum[0] * s.inv_d;
        const V off = P::of(-mu);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if ((v * TPR + lane) * VEC < s.D)   // the rest stays 0
#pragma unroll
                for (int i = 0; i < KP; ++i) xv[v][i] = add2(xv[v][i], off);
    }
    V acc = P::of(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < KP; ++i) acc = fma2(xv[v][i], xv[v][i], acc);
    float sq[1] = {P::sum(acc)};
    row_sum<TPR, 1>(sq, red, turn);
    rs = rsqrtf(sq[0] * s.inv_d + s.eps);   // within 2^-22 of its value
}


// GATE: x, z [, res] -> y; else x, res -> sum, y.
template <typename T, int TPR, int NV, int VEC, bool GATE, bool RES>
__global__ void __launch_bounds__(fwd_threads<TPR>())
block_norm_fwd_kernel(const T *x, const T *z, const T *res, const float *__restrict__ w, const float *__restrict__ b,
                      T *sum, T *y, float *__restrict__ mean, float *__restrict__ rstd, NormShape s, float scale,
                      int rms, int act) {
    constexpr int kThreads = fwd_threads<TPR>(), kTensors = 1 + GATE + RES;
    __shared__ float red[2][1][32];
    int turn = 0;
    Place p(TPR, s);
    constexpr int kDepth = VEC > 1 ? ring_depth<NV, kTensors>() : 2;
    extern __shared__ uint4 ring[];
    using Stream = RowStream<T, kThreads, TPR, NV, VEC>;
    auto open = [&](const T *t, int k) {
        Stream st{};
        st.p = t + p.row * s.D + p.lane * VEC;
        st.step = p.row_step * s.D;
        st.ring = ring + k * kDepth * NV * kThreads + threadIdx.x;
        st.p0 = t;
        return st;
    };
    Stream xs = open(x, 0), zs = open(GATE ? z : x, GATE ? 1 : 0), rs_ = open(RES ? res : x, RES ? 1 + GATE : 0);
    auto ask = [&](int slot, bool on) {
        xs.ask(slot, p.lane, s.D, on);
        if constexpr (GATE) zs.ask(slot, p.lane, s.D, on);
        if constexpr (RES) rs_.ask(slot, p.lane, s.D, on);
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) ask(i, p.mine && p.m + i * p.step < s.sets);
    // paired instructions: 32768 rows x 2048 95 us, single ones 98.5; with a gate 72 and 65 (524288 x 128),
    // whose exponentials come one by one
    using P = Pairs<VEC, (VEC > 1 && !GATE)>;
    using V = typename P::type;
    constexpr int kP = P::count;
    V wv[NV][kP], bv[NV][kP];
    load_affine<P, NV, VEC, TPR>(w, b, p, s, wv, bv);
    // every thread of the block takes the same number of steps (the sums synchronise)
    int slot = 0;
    for (int64_t m0 = p.m - p.ri; m0 < s.sets; m0 += p.step, p.m += p.step, p.row += p.row_step) {
        const bool on = p.mine && p.m < s.sets;
        ask(slot == 0 ? kDepth - 1 : slot - 1, p.mine && p.m + (kDepth - 1) * p.step < s.sets);
        copies_wait<kDepth - 1>();
        typename Piece<T, VEC>::type rx[NV], rz[NV], rr[NV];
        xs.read(slot, rx);
        if constexpr (GATE) zs.read(slot, rz);
        if constexpr (RES) rs_.read(slot, rr);
        slot = slot == kDepth - 1 ? 0 : slot + 1;
        V xv[NV][kP];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float xe[VEC];
            widen<T, VEC>(rx[v], xe);
            if constexpr (!GATE) {
                float re[VEC];
                widen<T, VEC>(rr[v], re);
#pragma unroll
                for (int i = 0; i < VEC; ++i) xe[i] = rounded<T>(fmaf(scale, xe[i], re[i]));
                const int c = (v * TPR + p.lane) * VEC;
                if (on && c < s.D) store_n<T, VEC>(sum + p.row * s.D + c, xe);
            }
#pragma unroll
            for (int i = 0; i < kP; ++i) xv[v][i] = P::at(xe, i);
        }
        float mu, rs;
        row_stats<P, TPR, NV, VEC, kP, V>(xv, p.lane, s, rms, red, turn, mu, rs);
        if (on) {
            const V rs2 = P::of(rs), scale2 = P::of(scale);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + p.lane) * VEC;
                float o[VEC], ze[VEC], re[VEC];
                if constexpr (GATE) widen<T, VEC>(rz[v], ze);
                if constexpr (GATE && RES) widen<T, VEC>(rr[v], re);
#pragma unroll
                for (int i = 0; i < kP; ++i) {
                    V n = fma2(mul2(xv[v][i], rs2), wv[v][i], bv[v][i]);
                    if constexpr (GATE) {
                        const V z = P::at(ze, i);
                        V g = sigmoid_of<sizeof(T) == 4>(z);
                        if (act == GDR_ACT_SILU) g = mul2(g, z);
                        g = mul2(scale2, g);
                        n = RES ? fma2(n, g, P::at(re, i)) : mul2(n, g);
                    }
                    P::put(o, i, n);
                }
                if (c < s.D) store_n<T, VEC>(y + p.row * s.D + c, o);
            }
            if (p.lane == 0) {
                if (mean) mean[p.row] = mu;
                if (rstd) rstd[p.row] = rs;
            }
        }
    }
}

template <typename T, bool GATE, bool RES>
cudaError_t fwd_t(const void *x, const void *z, const void *res, const float *w, const float *b, void *sum, void *y,
                  float *mean, float *rstd, const BlockNorm &bn, int sms, cudaStream_t stream) {
    const bool pieces = in_pieces(bn.D, sizeof(T), {x, z, res, sum, y});
    const NormPick p = pick_block(bn.D, sizeof(T), pieces, GATE);
    const NormGrid n = norm_grid(p, bn.rows, bn.G, bn.D, bn.eps, sms, 256);
    return with_layout<T, true>(p, [&](auto tpr, auto nv, auto vec) {
        auto kern = block_norm_fwd_kernel<T, tpr(), nv(), vec(), GATE, RES>;
        constexpr int kTensors = 1 + GATE + RES;
        const int smem = vec() > 1 ? kTensors * ring_depth<nv(), kTensors>() * n.threads * 16 * nv() : 0;
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
        ProfScope prof(stream, GATE ? "norm_gate_fwd_kernel" : "add_norm_fwd_kernel");
        kern<<<n.grid, n.threads, smem, stream>>>((const T *)x, (const T *)z, (const T *)res, w, b, (T *)sum, (T *)y, mean,
                                                  rstd, n.s, bn.scale, bn.kind == GDR_NORM_RMS, bn.act);
        count_launch();
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_add_norm_fwd(const void *x, const void *res, const float *w, const float *b, void *sum, void *y,
                                float *mean, float *rstd, const BlockNorm &n, gdr_dtype_t dtype, int sms,
                                cudaStream_t stream) {
    return dtype == GDR_BF16
               ? fwd_t<__nv_bfloat16, false, true>(x, nullptr, res, w, b, sum, y, mean, rstd, n, sms, stream)
               : fwd_t<float, false, true>(x, nullptr, res, w, b, sum, y, mean, rstd, n, sms, stream);
}

cudaError_t launch_norm_gate_fwd(const void *x, const void *z, const float *w, const float *b, const void *res, void *y,
                                 float *mean, float *rstd, const BlockNorm &n, gdr_dtype_t dtype, int sms,
                                 cudaStream_t stream) {
    if (dtype == GDR_BF16)
        return res ? fwd_t<__nv_bfloat16, true, true>(x, z, res, w, b, nullptr, y, mean, rstd, n, sms, stream)
                   : fwd_t<__nv_bfloat16, true, false>(x, z, nullptr, w, b, nullptr, y, mean, rstd, n, sms, stream);
    return res ? fwd_t<float, true, true>(x, z, res, w, b, nullptr, y, mean, rstd, n, sms, stream)
               : fwd_t<float, true, false>(x, z, nullptr, w, b, nullptr, y, mean, rstd, n, sms, stream);
}

}  // namespace gdr
