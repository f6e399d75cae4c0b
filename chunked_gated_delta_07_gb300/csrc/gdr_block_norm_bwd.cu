// gdr_block_norm_bwd.cu -- gradients of the norms around a block (gdr_block_norm.cuh), from the
// forward's statistics.  With vh = (v - mu) s and n = w dN, dN the gradient of N's output,
//     through(n) = s (n - [mean(n)] - vh mean(n vh))            [layer norm alone]
//     add_norm:   dN = dy,  dresidual = dr + through(n),  dx = scale dresidual
//     norm_gate:  dN = scale dy act(z),  dx = through(n),  dz = scale dy (vh w + b) act'(z)
//     dw = sum_r dN vh,  db = sum_r dN
// Each tensor crosses HBM once, which bounds rows that a warp holds (128 columns, below); wider ones have a
// barrier of the block to each row, with three blocks on an SM (norm_gate 16384 x 2048 bf16: 79 us, its
// floor is 50).  Rows in registers and inputs through a ring as in the layer norm's
// backward pass, and as there the weights' sums stay in registers, dbias's also where it is not wanted,
// one partial sum per block, added in a fixed order by a second kernel.
#include "gdr_block_norm.cuh"

namespace gdr {
namespace {

using namespace norm;

// Threads of a block, and of an SM, as registers allow: a row's 8 elements of three tensors, the
// weights and both sums (524288 rows x 128 norm_gate: 512 threads an SM 131 us, 768 121, 1024 141 with
// spills; 8191 rows x 2048 add_norm: 35, 35, 41).
//
// Measured (bf16): norm_gate 524288 x 128 with 16 weight rows 121 to 124 us, 5.5 TB/s, 82% of a copy's
// rate; add_norm 8191 x 2048 35 us, 4.8 TB/s, 72% (8 us of it the sum of the partials).
constexpr int kLeast = 256, kPerSm = 768;
template <int TPR> constexpr int block_threads() { return TPR > kLeast ? TPR : kLeast; }
template <int TPR> constexpr int block_per_sm() { return block_threads<TPR>() > kPerSm ? block_threads<TPR>() : kPerSm; }
template <int TPR, int NV, int TENSORS> constexpr int block_depth() {
    constexpr int d = ring_depth<NV, TENSORS, block_per_sm<TPR>()>();
    return d > 0 ? d : 1;
}

// GATE: dy, v = x, z [b] -> dx, dz; else dy, v = r [, dr] -> dx (may be null), dres.
template <typename T, int TPR, int NV, int VEC, bool GATE, bool THREE>
__global__ void __launch_bounds__(block_threads<TPR>(), VEC > 1 ? block_per_sm<TPR>() / block_threads<TPR>() : 1)
block_norm_bwd_kernel(const T *dy, const T *val, const T *third, const float *__restrict__ mean,
                      const float *__restrict__ rstd, const float *__restrict__ w, const float *__restrict__ b, T *dx,
                      T *dother, float *__restrict__ part, NormShape s, float scale, int rms, int act) {
    constexpr int kThreads = block_threads<TPR>(), kTensors = 2 + THREE;
    __shared__ float red[2][2][32];
    let_next_start();
    int turn = 0;
    Place p(TPR, s);
    constexpr int kDepth = VEC > 1 ? block_depth<TPR, NV, kTensors>() : 2;
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
    Stream ds = open(dy, 0), vs = open(val, 1), ts = open(THREE ? third : val, THREE ? 2 : 1);
    auto ask = [&](int slot, bool on) {
        ds.ask(slot, p.lane, s.D, on);
        vs.ask(slot, p.lane, s.D, on);
        if constexpr (THREE) ts.ask(slot, p.lane, s.D, on);
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) ask(i, p.mine && p.m + i * p.step < s.sets);
    auto stats = [&](int64_t m, int64_t row, float &mu, float &rs) {
        const bool on = p.mine && m < s.sets;
        mu = on && mean ? mean[row] : 0.f;
        rs = on ? rstd[row] : 0.f;
    };
    float mu, rs;
    stats(p.m, p.row, mu, rs);
    using P = Pairs<VEC>;
    using V = typename P::type;
    constexpr int kP = P::count;
    V wv[NV][kP], bv[NV][kP], aw[NV][kP], ab[NV][kP];
    load_affine<P, NV, VEC, TPR>(w, GATE ? b : nullptr, p, s, wv, bv);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < kP; ++i) aw[v][i] = ab[v][i] = P::of(0.f);
    const V scale2 = P::of(scale);
    int slot = 0;
    for (int64_t m0 = p.m - p.ri; m0 < s.sets; m0 += p.step, p.m += p.step, p.row += p.row_step) {
        const bool on = p.mine && p.m < s.sets;
        ask(slot == 0 ? kDepth - 1 : slot - 1, p.mine && p.m + (kDepth - 1) * p.step < s.sets);
        float mu1, rs1;
        stats(p.m + p.step, p.row + p.row_step, mu1, rs1);
        copies_wait<kDepth - 1>();
        typename Piece<T, VEC>::type rv[NV], rd[NV], rt[NV];
        vs.read(slot, rv);
        ds.read(slot, rd);
        if constexpr (THREE) ts.read(slot, rt);
        slot = slot == kDepth - 1 ? 0 : slot + 1;
        // dy is 0 where there is no row or column, so that nothing there counts
        V xv[NV][kP], dv[NV][kP], sum0 = P::of(0.f), sum1 = P::of(0.f);   // of n, of n vh
        const V rs2 = P::of(rs), off = P::of(-mu);   // the mean comes off first: x rs - mu rs would round mu rs
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + p.lane) * VEC;
            const bool in = on && c < s.D;
            float xe[VEC], de[VEC], ze[VEC], oz[VEC];
            widen<T, VEC>(rv[v], xe);
            widen<T, VEC>(rd[v], de);
            if constexpr (GATE) widen<T, VEC>(rt[v], ze);
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                const V xh = mul2(add2(P::at(xe, i), off), rs2);
                V d = P::at(de, i);
                if constexpr (GATE) {
                    const V z = P::at(ze, i), g = sigmoid_of<sizeof(T) == 4>(z), n = fma2(xh, wv[v][i], bv[v][i]);
                    // act' = g (1 + z (1 - g)) (silu) or g (1 - g); 1 - g is 0 where g is 1, however large z is
                    const V left = fma2(g, P::of(-1.f), P::of(1.f));
                    const V a = act == GDR_ACT_SILU ? mul2(z, g) : g;
                    const V slope = mul2(g, act == GDR_ACT_SILU ? fma2(z, left, P::of(1.f)) : left);
                    d = mul2(scale2, d);
                    P::put(oz, i, mul2(mul2(d, n), slope));
                    d = mul2(d, a);
                }
                aw[v][i] = fma2(d, xh, aw[v][i]);
                ab[v][i] = add2(ab[v][i], d);
                d = mul2(d, wv[v][i]);
                sum0 = add2(sum0, d);
                sum1 = fma2(d, xh, sum1);
                xv[v][i] = xh;
                dv[v][i] = d;
            }
            if constexpr (GATE)
                if (in) store_n<T, VEC>(dother + p.row * s.D + c, oz);
        }
        float sum[2] = {P::sum(sum0), P::sum(sum1)};
        row_sum<TPR, 2>(sum, red, turn);
        // rs (dv - c1 - xh c2)
        const V k1 = P::of(rms ? 0.f : -rs * sum[0] * s.inv_d), k2 = P::of(-rs * sum[1] * s.inv_d);
        if (on) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + p.lane) * VEC;
                if (c >= s.D) continue;
                float o[VEC];
                if constexpr (GATE) {
#pragma unroll
                    for (int i = 0; i < kP; ++i) P::put(o, i, fma2(dv[v][i], rs2, fma2(xv[v][i], k2, k1)));
                    store_n<T, VEC>(dx + p.row * s.D + c, o);
                } else {
                    float te[VEC];
                    if constexpr (THREE) widen<T, VEC>(rt[v], te);
#pragma unroll
                    for (int i = 0; i < kP; ++i)
                        P::put(o, i, fma2(dv[v][i], rs2, fma2(xv[v][i], k2, THREE ? add2(k1, P::at(te, i)) : k1)));
                    store_n<T, VEC>(dother + p.row * s.D + c, o);
                    if (dx) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) o[i] *= scale;
                        store_n<T, VEC>(dx + p.row * s.D + c, o);
                    }
                }
            }
        }
        mu = mu1;
        rs = rs1;
    }
    // no copy of this thread's may still be on its way into the ring: those asked for past the
    // last row fill it with zeros, and its memory is taken for the groups' sums below
    copies_wait<0>();
    if (!part) return;
    float sw[NV][VEC], sb[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            P::put(sw[v], i, aw[v][i]);
            P::put(sb[v], i, ab[v][i]);
        }
    block_partials<kThreads, TPR, NV, VEC>(sw, sb, part, (float *)ring, p.gi, p.ri, p.lane, p.g, p.mine, s);
}

template <typename T, bool GATE, bool THREE>
cudaError_t bwd_t(const void *dy, const void *val, const void *third, const float *mean, const float *rstd, const float *w,
                  const float *b, void *dx, void *dother, float *dw, float *db, const BlockNorm &bn, int sms, float *scratch,
                  cudaStream_t stream) {
    const NormPick p = pick_block(bn.D, sizeof(T), in_pieces(bn.D, sizeof(T), {dy, val, third, dx, dother}), true);
    const NormGrid n = norm_grid(p, bn.rows, bn.G, bn.D, 0.f, sms, kLeast, kPerSm);
    float *part = dw || db ? scratch : nullptr;
    const cudaError_t err = with_layout<T, true>(p, [&](auto tpr, auto nv, auto vec) {
        auto kern = block_norm_bwd_kernel<T, tpr(), nv(), vec(), GATE, THREE>;
        constexpr int kTensors = 2 + THREE;
        const int smem = std::max(vec() > 1 ? kTensors * block_depth<tpr(), nv(), kTensors>() * n.threads * 16 * nv() : 0,
                                  n.threads * 4 * nv() * vec());
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess) return err;
        ProfScope prof(stream, GATE ? "norm_gate_bwd_kernel" : "add_norm_bwd_kernel");
        kern<<<n.grid, n.threads, smem, stream>>>((const T *)dy, (const T *)val, (const T *)third, mean, rstd, w, b,
                                                  (T *)dx, (T *)dother, part, n.s, bn.scale, bn.kind == GDR_NORM_RMS,
                                                  bn.act);
        count_launch();
        return cudaGetLastError();
    });
    if (err != cudaSuccess || !part) return err;
    return launch_norm_sum(part, dw, db, (int)n.grid.y, (int64_t)bn.G * bn.D, stream);
}

}  // namespace

size_t block_norm_bwd_scratch_bytes(int64_t rows, int G, int D, gdr_dtype_t dtype, int sms) {
    const size_t es = dtype == GDR_BF16 ? 2 : 4;
    size_t need = 0;   // whichever layout the pointers' alignment allows
    for (bool pieces : {true, false})
        need = std::max(need, sizeof(float) * 2 * (size_t)G * D *
                                  norm_grid(pick_block(D, es, pieces, true), rows, G, D, 0.f, sms, kLeast, kPerSm).grid.y);
    return need;
}

cudaError_t launch_add_norm_bwd(const void *dy, const void *dsum, const void *sum, const float *mean, const float *rstd,
                                const float *w, void *dx, void *dres, float *dw, float *db, const BlockNorm &n,
                                gdr_dtype_t dtype, int sms, float *scratch, cudaStream_t stream) {
    if (dtype == GDR_BF16)
        return dsum ? bwd_t<__nv_bfloat16, false, true>(dy, sum, dsum, mean, rstd, w, nullptr, dx, dres, dw, db, n, sms,
                                                        scratch, stream)
                    : bwd_t<__nv_bfloat16, false, false>(dy, sum, nullptr, mean, rstd, w, nullptr, dx, dres, dw, db, n,
                                                         sms, scratch, stream);
    return dsum ? bwd_t<float, false, true>(dy, sum, dsum, mean, rstd, w, nullptr, dx, dres, dw, db, n, sms, scratch, stream)
                : bwd_t<float, false, false>(dy, sum, nullptr, mean, rstd, w, nullptr, dx, dres, dw, db, n, sms, scratch,
                                             stream);
}

cudaError_t launch_norm_gate_bwd(const void *dy, const void *x, const void *z, const float *mean, const float *rstd,
                                 const float *w, const float *b, void *dx, void *dz, float *dw, float *db,
                                 const BlockNorm &n, gdr_dtype_t dtype, int sms, float *scratch, cudaStream_t stream) {
    return dtype == GDR_BF16
               ? bwd_t<__nv_bfloat16, true, true>(dy, x, z, mean, rstd, w, b, dx, dz, dw, db, n, sms, scratch, stream)
               : bwd_t<float, true, true>(dy, x, z, mean, rstd, w, b, dx, dz, dw, db, n, sms, scratch, stream);
}

}  // namespace gdr
