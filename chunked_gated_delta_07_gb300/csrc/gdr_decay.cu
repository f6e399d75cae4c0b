// gdr_decay.cu -- linear attention with one constant decay per head, token by token on
// the CUDA cores, and the chaining of segment states.
//
// decay_rec_kernel runs one pass (gdr_decay.cuh) in its recurrent form.  The columns of
// the state S (kd x vd) are independent, so a block owns one (segment, head, 64-column
// slice) and keeps it in registers, 8 x 8 elements per thread, while the tokens stream
// through shared memory in tiles of 16.  Per token a thread does 64 updates and 64
// products for out = S^T a, whose sum over kd is a halving exchange over the kd / 8 lanes
// that share columns.  The arithmetic is fp32 throughout; the pass is bound by the CUDA
// cores (2 kd vd fused multiply-adds per token and head against 2 kd + 2 vd elements moved).
#include <algorithm>

#include "gdr_decay.cuh"

namespace gdr {

GDR_DEBUG_TU()

namespace {

constexpr int kTb = 16;     // tokens per staged tile
constexpr int kCols = 64;   // state columns per block

template <typename T, int KD, bool REV, bool OUT>
__global__ void __launch_bounds__(KD)
decay_rec_kernel(const DecayGeom g, const DecayPass p) {
    constexpr int kLanes = KD / 8;   // threads along kd; 8 threads along the columns
    constexpr unsigned kFull = 0xffffffffu;
    __shared__ __align__(16) float bs[kTb][KD];
    __shared__ __align__(16) float as[OUT ? kTb : 1][KD];
    __shared__ __align__(16) float cs[kTb][kCols];
    __shared__ float os[OUT ? kTb : 1][kCols];
    __shared__ float pw[kTb][2];   // lam^j, lam^-j
    const int slices = p.vd / kCols;
    const int e0 = (int)(blockIdx.x % slices) * kCols;
    const int64_t sh = blockIdx.x / slices;
    const int h = (int)(sh % g.H);
    DecaySeg seg;
    if (!decay_segment(g, sh / g.H, seg)) return;
    if (!OUT && (REV ? seg.first : seg.last)) return;   // no boundary behind it
    if (!GDR_INBOUNDS(seg.t0 >= 0 && seg.t1 <= g.T_total && (!p.slots || seg.slot <= g.max_slots))) return;
    const float gd = decay_log(g.log_decay, h);
    int64_t t0 = seg.t0, t1 = seg.t1;
    if (!OUT) {
        const int64_t reach = decay_reach(gd, t1 - t0);
        if (REV) t1 = t0 + reach; else t0 = t1 - reach;
    }
    const int64_t ntok = t1 - t0;
    // Inside a block of nb tokens the state is kept without its decay: with j tokens of the
    // block behind it, S = lam^j S^, S^ += lam^-j b c^T and out = (lam^j a)^T S^, and lam^nb
    // enters the state once per block.  That saves a third of the instructions and keeps the
    // powers exact: lam itself rounds to 24 bits, an error that a product of n of them
    // multiplies by n.  Blocks are
    // whole tiles while lam^-15 stays in range, else single tokens.  A forward pass decays the
    // state before its first token too, a reversed one after its last.
    const int nb = gd >= -4.f ? kTb : 1;
    const DecayFactor step(gd * (float)nb);
    const int tid = threadIdx.x, dl = tid % kLanes, eg = tid / kLanes;
    // the thread's elements: kd index 4 dl + (u & 3) + (u >> 2) KD / 2, column e0 + 8 eg + j
    float s[8][8];
    const float *in = decay_state_in(p, seg, g.H, h);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int d = 4 * dl + (u & 3) + (u >> 2) * (KD / 2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = e0 + 8 * eg + j;
            s[u][j] = in ? in[p.transposed ? (int64_t)e * KD + d : (int64_t)d * p.vd + e] : 0.f;
        }
    }
    auto decay = [&](const DecayFactor &f) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[u][j] = f(s[u][j]);
    };
    if (!REV && ntok > 0) decay(DecayFactor(gd));
    if (tid < kTb) {
        const float e = nb > 1 ? gd * (float)tid : 0.f;
        pw[tid][0] = expf(e);
        pw[tid][1] = expf(-e);
    }
    __syncthreads();
    const T *A = (const T *)p.a, *B = (const T *)p.b, *C = (const T *)p.c;
    T *O = (T *)p.out;
    for (int64_t tb = 0; tb < ntok; tb += kTb) {
        const int nr = (int)min((int64_t)kTb, ntok - tb);
        if (tb && nb > 1) decay(step);
        // token of the tile's row r, in the order of the pass
        auto row_of = [&](int r) { return (REV ? t1 - 1 - (tb + r) : t0 + tb + r) * g.H + h; };
        for (int i = tid; i < nr * KD; i += KD) {
            const int64_t at = row_of(i / KD) * KD + i % KD;
            bs[i / KD][i % KD] = to_f32(B[at]);
            if (OUT) as[i / KD][i % KD] = to_f32(A[at]) * (p.s_out * pw[i / KD][0]);
        }
        for (int i = tid; i < nr * kCols; i += KD)
            cs[i / kCols][i % kCols] = to_f32(C[row_of(i / kCols) * p.vd + e0 + i % kCols]) * (p.s_upd * pw[i / kCols][1]);
        __syncthreads();
#pragma unroll 2
        for (int r = 0; r < nr; ++r) {
            if (nb == 1 && tb + r) decay(step);
            float bv[8], cv[8], av[8], o[8];
            *(float4 *)&bv[0] = *(const float4 *)&bs[r][4 * dl];
            *(float4 *)&bv[4] = *(const float4 *)&bs[r][4 * dl + KD / 2];
            *(float4 *)&cv[0] = *(const float4 *)&cs[r][8 * eg];
            *(float4 *)&cv[4] = *(const float4 *)&cs[r][8 * eg + 4];
            if (OUT) {
                *(float4 *)&av[0] = *(const float4 *)&as[r][4 * dl];
                *(float4 *)&av[4] = *(const float4 *)&as[r][4 * dl + KD / 2];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[u][j] = fmaf(bv[u], cv[j], s[u][j]);
                    if (OUT) o[j] = fmaf(av[u], s[u][j], o[j]);
                }
            if (OUT) {
                // sum over the kLanes threads of the columns: each exchange halves the
                // columns a thread carries; lane bits give the column it ends with
                int col = 0, lanes = kLanes;
#pragma unroll
                for (int n = 4; n; n >>= 1) {
                    lanes >>= 1;
                    const bool up = dl & lanes;
#pragma unroll
                    for (int j = 0; j < n; ++j) {
                        const float send = up ? o[j] : o[j + n];
                        o[j] = (up ? o[j + n] : o[j]) + __shfl_xor_sync(kFull, send, lanes);
                    }
                    if (up) col += n;
                }
                if (kLanes == 16) o[0] += __shfl_xor_sync(kFull, o[0], 1);
                if (kLanes == 8 || !(dl & 1)) os[r][8 * eg + col] = o[0];
            }
        }
        __syncthreads();
        if (OUT)
            for (int i = tid; i < nr * kCols; i += KD)
                O[row_of(i / kCols) * p.vd + e0 + i % kCols] = from_f32<T>(os[i / kCols][i % kCols]);
    }
    float *to = decay_state_out(p, seg, g.H, h);
    if (!to) return;
    if (ntok > 0) decay(DecayFactor(gd * (float)((nb > 1 ? (ntok - 1) % kTb : 0) + (REV ? 1 : 0))));
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int d = 4 * dl + (u & 3) + (u >> 2) * (KD / 2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = e0 + 8 * eg + j;
            to[p.transposed ? (int64_t)e * KD + d : (int64_t)d * p.vd + e] = s[u][j];
        }
    }
}

// A few tokens of every sequence, the state updated in place.  A block owns 64 columns of
// one (sequence, head)'s state: 256 threads hold kd / 16 rows x 4 columns each as float4,
// all loaded before anything else (32 KB a block in flight at kd = 128), so that the
// pass is bound by the state's traffic, 2 x 4 kd vd bytes.  Sums over kd: a shuffle, then
// the 8 warps' partial sums through shared memory.
template <typename T, int KD>
__global__ void __launch_bounds__(256)
decay_step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                  const float *__restrict__ log_decay, float *__restrict__ state, T *__restrict__ out, int64_t Tn,
                  int H, int vd, float scale) {
    constexpr int kRows = KD / 16;
    __shared__ float ks[2][KD], qs[2][KD];
    __shared__ __align__(16) float vs[2][kCols];
    __shared__ __align__(16) float red[2][8][kCols];
    const int slices = vd / kCols;
    const int e0 = (int)(blockIdx.x % slices) * kCols;
    const int64_t nh = blockIdx.x / slices;
    const int64_t n = nh / H;
    const int h = (int)(nh % H);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c4 = (tid & 15) * 4, r0 = tid >> 4;   // first column; rows r0 + 16 u
    float4 *S = (float4 *)(state + (nh * KD + r0) * vd + e0 + c4);
    float4 s[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) s[u] = S[(int64_t)4 * u * vd];
    const DecayFactor decay(decay_log(log_decay, h));
    for (int64_t t = 0; t < Tn; ++t) {
        const int b = t & 1;
        const int64_t row = (n * Tn + t) * H + h;
        if (tid < KD) ks[b][tid] = to_f32(k[row * KD + tid]);
        else if (KD == 64 && tid < 2 * KD) qs[b][tid - KD] = to_f32(q[row * KD + tid - KD]) * scale;
        if (KD == 128 && tid >= KD) qs[b][tid - KD] = to_f32(q[row * KD + tid - KD]) * scale;
        if (tid < kCols) vs[b][tid] = to_f32(v[row * vd + e0 + tid]);
        __syncthreads();
        const float4 vv = *(const float4 *)&vs[b][c4];
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const float kd = ks[b][r0 + 16 * u], qd = qs[b][r0 + 16 * u];
            s[u] = make_float4(fmaf(kd, vv.x, decay(s[u].x)), fmaf(kd, vv.y, decay(s[u].y)),
                               fmaf(kd, vv.z, decay(s[u].z)), fmaf(kd, vv.w, decay(s[u].w)));
            o = make_float4(fmaf(qd, s[u].x, o.x), fmaf(qd, s[u].y, o.y), fmaf(qd, s[u].z, o.z),
                            fmaf(qd, s[u].w, o.w));
        }
        if (t == Tn - 1)
#pragma unroll
            for (int u = 0; u < kRows; ++u) S[(int64_t)4 * u * vd] = s[u];
        o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
        if (lane < 16) *(float4 *)&red[b][warp][c4] = o;
        __syncthreads();
        if (tid < kCols) {
            float a = red[b][0][tid];
#pragma unroll
            for (int w = 1; w < 8; ++w) a += red[b][w][tid];
            out[row * vd + e0 + tid] = from_f32<T>(a);
        }
    }
}

// cur = s0; per segment in the order of the pass: cur = lam^len cur + its local sum, the
// state that enters the next segment, written over the sum.  A block takes 1024 elements
// of one (sequence, head).
__global__ void __launch_bounds__(256)
decay_combine_kernel(const DecayGeom g, const DecayPass p) {
    const int64_t st = (int64_t)p.kd * p.vd;
    const int parts = (int)(st / 1024);
    const int64_t at = (blockIdx.x % parts) * 1024 + 4 * threadIdx.x;
    const int64_t nh = blockIdx.x / parts;
    const int h = (int)(nh % g.H), n = (int)(nh / g.H);
    int64_t base, cnt, len;
    if (g.dense) {
        base = n * g.segs_per_seq;
        cnt = g.segs_per_seq;
        len = g.T_per;
    } else {
        base = g.p.seg_base[n];
        cnt = g.p.seg_base[n + 1] - base;
        len = g.p.seq_start[n + 1] - g.p.seq_start[n];
    }
    if (cnt < 2 || !GDR_INBOUNDS(base - n + cnt - 1 <= g.max_slots)) return;
    const float gd = decay_log(g.log_decay, h);
    const DecayFactor full(gd * (float)g.seg_tokens);
    float4 cur = p.s0 ? *(const float4 *)&p.s0[nh * st + at] : make_float4(0.f, 0.f, 0.f, 0.f);
    float *slots = p.slots + ((base - n) * g.H + h) * st + at;
#pragma unroll 4
    for (int64_t i = 0; i < cnt - 1; ++i) {
        // reversed: the last segment, which may be short, comes first
        const DecayFactor f = p.rev && i == 0 ? DecayFactor(gd * (float)(len - (cnt - 1) * g.seg_tokens)) : full;
        float4 *sp = (float4 *)&slots[(p.rev ? cnt - 2 - i : i) * g.H * st];
        const float4 x = *sp;
        cur = make_float4(f(cur.x) + x.x, f(cur.y) + x.y, f(cur.z) + x.z, f(cur.w) + x.w);
        *sp = cur;
    }
}

template <typename T, int KD>
cudaError_t rec_t(const DecayGeom &g, const DecayPass &p, cudaStream_t stream) {
    const int64_t blocks = g.max_segs * g.H * (p.vd / kCols);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (blocks == 0) return cudaSuccess;
    ProfScope prof(stream, p.local ? "decay_rec_kernel (local)" : "decay_rec_kernel");
    const unsigned n = (unsigned)blocks;
    if (!p.local) {
        if (p.rev) decay_rec_kernel<T, KD, true, true><<<n, KD, 0, stream>>>(g, p);
        else decay_rec_kernel<T, KD, false, true><<<n, KD, 0, stream>>>(g, p);
    } else {
        if (p.rev) decay_rec_kernel<T, KD, true, false><<<n, KD, 0, stream>>>(g, p);
        else decay_rec_kernel<T, KD, false, false><<<n, KD, 0, stream>>>(g, p);
    }
    count_launch();
    return cudaGetLastError();
}

template <typename T>
cudaError_t step_t(const void *q, const void *k, const void *v, const float *log_decay, float *state, void *out,
                   int N, int64_t Tn, int H, int dk, int dv, float scale, cudaStream_t stream) {
    const int64_t blocks = (int64_t)N * H * (dv / kCols);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    ProfScope prof(stream, "decay_step_kernel");
    auto kern = dk == 128 ? decay_step_kernel<T, 128> : decay_step_kernel<T, 64>;
    kern<<<(unsigned)blocks, 256, 0, stream>>>((const T *)q, (const T *)k, (const T *)v, log_decay, state, (T *)out,
                                               Tn, H, dv, scale);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_step(const void *q, const void *k, const void *v, const float *log_decay, float *state,
                              void *out, gdr_dtype_t dtype, int N, int64_t T, int H, int dk, int dv, float scale,
                              cudaStream_t stream) {
    return dtype == GDR_BF16 ? step_t<__nv_bfloat16>(q, k, v, log_decay, state, out, N, T, H, dk, dv, scale, stream)
                             : step_t<float>(q, k, v, log_decay, state, out, N, T, H, dk, dv, scale, stream);
}

cudaError_t launch_decay_rec(const DecayGeom &g, const DecayPass &p, gdr_dtype_t dtype, cudaStream_t stream) {
    if (dtype == GDR_BF16)
        return p.kd == 128 ? rec_t<__nv_bfloat16, 128>(g, p, stream) : rec_t<__nv_bfloat16, 64>(g, p, stream);
    return p.kd == 128 ? rec_t<float, 128>(g, p, stream) : rec_t<float, 64>(g, p, stream);
}

cudaError_t launch_decay_combine(const DecayGeom &g, const DecayPass &p, cudaStream_t stream) {
    const int64_t blocks = (int64_t)g.N * g.H * ((int64_t)p.kd * p.vd / 1024);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    ProfScope prof(stream, "decay_combine_kernel");
    decay_combine_kernel<<<(unsigned)blocks, 256, 0, stream>>>(g, p);
    count_launch();
    return cudaGetLastError();
}

}  // namespace gdr
