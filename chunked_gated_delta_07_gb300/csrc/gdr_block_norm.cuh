// gdr_block_norm.cuh -- the norms around a block, with what stands next to them in one pass:
//     add_norm (in front):  r = residual + scale x,  y = N(r)
//     norm_gate (behind):   y = [residual +] scale N(x) act(z)
//     N(v) = vh w + b,  vh = (v - mu) s,  s = (mean((v - mu)^2) + eps)^{-1/2},  mu = mean(v) or 0 (rms)
#pragma once

#include "gdr_norm.cuh"
#include "gdr_pairs.cuh"

namespace gdr {

struct BlockNorm {
    int64_t rows;
    int G, D;
    float scale, eps;
    gdr_norm_kind_t kind;
    gdr_act_t act;
};

size_t block_norm_bwd_scratch_bytes(int64_t rows, int G, int D, gdr_dtype_t dtype, int sms);
cudaError_t launch_add_norm_fwd(const void *x, const void *res, const float *w, const float *b, void *sum, void *y,
                                float *mean, float *rstd, const BlockNorm &n, gdr_dtype_t dtype, int sms,
                                cudaStream_t stream);
// dx may be null (not wanted)
cudaError_t launch_add_norm_bwd(const void *dy, const void *dsum, const void *sum, const float *mean, const float *rstd,
                                const float *w, void *dx, void *dres, float *dw, float *db, const BlockNorm &n,
                                gdr_dtype_t dtype, int sms, float *scratch, cudaStream_t stream);
cudaError_t launch_norm_gate_fwd(const void *x, const void *z, const float *w, const float *b, const void *res, void *y,
                                 float *mean, float *rstd, const BlockNorm &n, gdr_dtype_t dtype, int sms,
                                 cudaStream_t stream);
cudaError_t launch_norm_gate_bwd(const void *dy, const void *x, const void *z, const float *mean, const float *rstd,
                                 const float *w, const float *b, void *dx, void *dz, float *dw, float *db,
                                 const BlockNorm &n, gdr_dtype_t dtype, int sms, float *scratch, cudaStream_t stream);

#ifdef __CUDACC__
namespace norm {

// As the layer norm's, but of single elements rows of up to 4096 go to the smallest power of two of
// threads with 8 each, there every other one (16384 rows x 2047 bf16 on 256 threads against 512:
// add_norm 175 -> 66 us, its backward 147 -> 86, norm_gate 140 -> 77, its backward 169 -> 107; from 2049
// columns on both take 512, and 256 threads of 16 were not measured there: 11000 rows x 3001 add_norm 128 us,
// norm_gate 105).  Where `wide` says so, rows of 4097 to 8192 go to 1024 threads: three tensors' 16 elements do
// not fit into a thread (8192 rows x 4097 bf16: norm_gate 157 -> 147 us, its backward 373 -> 290, add_norm's
// 287 -> 245; add_norm itself 87 -> 121, which keeps 512).
inline NormPick pick_block(int D, size_t es, bool pieces, bool wide) {
    if (!pieces && D <= 4096) {
        int tpr = 8;
        while (tpr * 8 < D) tpr *= 2;
        return {tpr, 8, 1};
    }
    if (!pieces && wide && D <= 8192) return {1024, 8, 1};
    return pick_layout(D, es, pieces);
}

// sigmoid(z): within 2^-21 of its value for fp32 tensors; for bf16 ones, whose exponential and division are
// the fast ones, within (4 + 1.2 |z|) 2^-23, far below a step of bf16.  exp(-z) may be inf, which
// gives 0: below z = -88.7, for bf16 tensors below -87.3, where the value is below 2^-126.
template <bool FINE> __device__ __forceinline__ float sigmoid_of(float z) {
    if constexpr (FINE) return __frcp_rn(1.f + expf(-z));
    return __fdividef(1.f, 1.f + __expf(-z));
}
template <bool FINE> __device__ __forceinline__ float2 sigmoid_of(float2 z) {
    return make_float2(sigmoid_of<FINE>(z.x), sigmoid_of<FINE>(z.y));
}

template <typename T> __device__ __forceinline__ float rounded(float v) { return to_f32(from_f32<T>(v)); }

// The place of a thread of a block: its weight row g, its row set, the columns of its pieces.
struct Place {
    int lane, gi, ri, g;
    bool mine;
    int64_t step, row_step, m, row;
    __device__ __forceinline__ Place(int tpr, const NormShape &s) {
        const int sub = threadIdx.x / tpr;
        lane = threadIdx.x % tpr;
        gi = sub % s.gpb;
        ri = sub / s.gpb;
        g = blockIdx.x * s.gpb + gi;
        mine = ri < s.rpb && g < s.G;
        step = (int64_t)gridDim.y * s.rpb;
        row_step = step * s.G;
        m = (int64_t)blockIdx.y * s.rpb + ri;
        row = m * s.G + g;
    }
};

// The weight (1 without) and the bias (0 without) of a thread's columns.
template <typename P, int NV, int VEC, int TPR, typename V, int KP>
__device__ __forceinline__ void load_affine(const float *w, const float *b, const Place &pl, const NormShape &s,
                                            V (&wv)[NV][KP], V (&bv)[NV][KP]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float we[VEC], be[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (v * TPR + pl.lane) * VEC + i;
            const bool in = pl.mine && c < s.D;
            we[i] = in && w ? w[(int64_t)pl.g * s.D + c] : 1.f;
            be[i] = in && b ? b[(int64_t)pl.g * s.D + c] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            wv[v][i] = P::at(we, i);
            bv[v][i] = P::at(be, i);
        }
    }
}

}  // namespace norm
#endif

}  // namespace gdr
