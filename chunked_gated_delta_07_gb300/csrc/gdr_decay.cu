// gdr_decay.cu -- linear attention with one constant decay per head, token by token on
// the CUDA cores, and the chaining of segment states.
//
// decay_rec_kernel runs one pass (gdr_decay.cuh) in its recurrent form.  The columns of
// the state S (kd x vd) are independent, so a block owns one (segment, head, 64-column
// slice) and keeps it in registers, 4 x 8 elements per thread, while the tokens stream
// through shared memory in tiles of 16, the next tile's loads on their way.  Per token a thread
// does 32 updates and 32 products for out = S^T a, whose sum over kd is a halving exchange over
// the kd / 4 lanes that share columns.  The arithmetic is fp32 throughout.  Few blocks: bound by
// a token's chain of exchanges, 0.3 us a token (7 packed sequences, 5003 tokens of 2 heads x 64 in
// fp32, backward: 62 us in all).  Many: by issue slots, a quarter of the multiply-adds' rate
// (8 x 4096 tokens of 16 heads x 128 in fp32, forward: 2.2 ms, 0.41 of them the local pass).  8 x 8
// elements halve the exchanges, but the threads too: the packed call took 238 us with them and 86
// with 4 x 8.
#include <algorithm>
#include <type_traits>

#include "gdr_decay.cuh"

namespace gdr {

GDR_DEBUG_TU()

namespace {

// Exclusive sums of the sequences' segments (at least one each) over 1024 threads, each
// with a run of sequences; 32 sums of warps in one more.
__global__ void __launch_bounds__(1024)
decay_plan_kernel(const int32_t *__restrict__ cu, int N, int64_t T_total, int64_t seg_tokens,
                  int64_t *__restrict__ seq_start, int64_t *__restrict__ seg_base, unsigned long long *next,
                  int *status) {
    __shared__ int64_t sums[32];
    let_next_start();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (N + 1023) / 1024, n0 = min(N, tid * per), n1 = min(N, n0 + per);
    auto segments = [&](int64_t len) { return len > seg_tokens ? (len + seg_tokens - 1) / seg_tokens : 1; };
    int64_t mine = 0;
    bool bad = tid == 0 && (cu[0] != 0 || (int64_t)cu[N] != T_total);
    for (int n = n0; n < n1; ++n) {
        const int64_t len = (int64_t)cu[n + 1] - cu[n];
        bad |= len < 0;
        mine += segments(len);
    }
    int64_t at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += x;
    }
    if (lane == 31) sums[warp] = at;
    bad = __syncthreads_or(bad);
    int64_t before = lane < warp ? sums[lane] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    at += before - mine;
    if (tid < 2) next[tid] = 0;
    // bad offsets: an empty plan, every sequence without tokens or segments
    for (int n = n0; n < n1; ++n) {
        seq_start[n] = bad ? 0 : cu[n];
        seg_base[n] = bad ? 0 : at;
        at += segments((int64_t)cu[n + 1] - cu[n]);
    }
    if (tid == 1023) {
        seq_start[N] = bad ? 0 : T_total;
        seg_base[N] = bad ? 0 : at;
    }
    if (tid == 0 && bad) set_status(status, GDR_ERR_BAD_SEQLENS);
}

// Passes of one launch; blockIdx.y says which.
struct Passes {
    DecayPass p[kDecayMaxPasses];
};

constexpr int kTb = 16;     // tokens per staged tile
constexpr int kCols = 64;   // state columns per block

template <typename T, int KD, bool OUT>
__global__ void __launch_bounds__(2 * KD)
decay_rec_kernel(const DecayGeom g, const __grid_constant__ Passes passes) {
    const DecayPass &p = passes.p[blockIdx.y];
    constexpr int kThreads = 2 * KD;
    constexpr int kLanes = KD / 4;   // threads along kd, 4 rows each; 8 threads along the columns
    constexpr unsigned kFull = 0xffffffffu;
    __shared__ __align__(16) float bs[kTb][KD];
    __shared__ __align__(16) float as[OUT ? kTb : 1][KD];
    __shared__ __align__(16) float cs[kTb][kCols];
    __shared__ float os[OUT ? kTb : 1][kCols];
    __shared__ float pw[kTb][2];   // lam^j, lam^-j
    let_next_start();
    after_previous();
    const int vd = p.vd, slices = vd / kCols, H = g.H;
    if (blockIdx.x >= g.max_segs * H * slices) return;   // of a wider pass
    const int e0 = (int)(blockIdx.x % slices) * kCols;
    const int64_t sh = blockIdx.x / slices;
    const int h = (int)(sh % H);
    const bool rev = p.rev;
    DecaySeg seg;
    if (!decay_segment(g, sh / H, seg)) return;
    if (!OUT && (rev ? seg.first : seg.last)) return;   // no boundary behind it
    if (!GDR_INBOUNDS(seg.t0 >= 0 && seg.t1 <= g.T_total && (!p.slots || seg.slot <= g.max_slots))) return;
    const float gd = decay_log(g.log_decay, h);
    // (a local pass takes all of them too, however little the decay leaves of the early ones: a NaN
    // stays.  Leaving those out gained nothing up to 65536 tokens of one head, 8% with 16 heads.)
    const int64_t t0 = seg.t0, t1 = seg.t1, ntok = t1 - t0;
    // Inside a block of nb tokens the state is kept without its decay: with j tokens of the
    // block behind it, S = lam^j S^, S^ += lam^-j b c^T and out = (lam^j a)^T S^, and lam^nb
    // enters the state once per block.  That saves a third of the instructions and keeps the
    // powers exact: lam itself rounds to 24 bits, an error that a product of n of them
    // multiplies by n.  Blocks are whole tiles while lam^-15 costs no more than 2^22 of fp32's
    // range, else single tokens (8 x 4096 tokens of 16 heads, all so fast: 3.0 ms against 2.2).  A
    // forward pass decays the state before its first token too, a reversed one after its last.
    const int nb = gd >= -1.f ? kTb : 1;
    const DecayFactor step(gd * (float)nb);
    const int tid = threadIdx.x, dl = tid % kLanes, eg = tid / kLanes;
    // the thread's elements: row 4 dl + u of kd, column e0 + 8 eg + j
    float s[4][8];
    const float *in = decay_state_in(p, seg, H, h);
    if (!in) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[u][j] = 0.f;
    } else if (p.transposed) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 x = *(const float4 *)&in[(e0 + 8 * eg + j) * KD + 4 * dl];
            s[0][j] = x.x, s[1][j] = x.y, s[2][j] = x.z, s[3][j] = x.w;
        }
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *(float4 *)&s[u][j] = *(const float4 *)&in[(4 * dl + u) * vd + e0 + 8 * eg + j];
    }
    auto decay = [&](const DecayFactor &f) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[u][j] = f(s[u][j]);
    };
    if (!rev && ntok > 0) decay(DecayFactor(gd));
    if (tid < kTb) {
        const float e = nb > 1 ? gd * (float)tid : 0.f;
        pw[tid][0] = expf(e);
        pw[tid][1] = expf(-e);
    }
    // A tile's tokens in the order of the pass, as loaded: the next tile's are on their way
    // while one is computed
    constexpr int kPerB = kTb * KD / kThreads, kPerC = kTb * kCols / kThreads;
    const T *A = (const T *)p.a, *B = (const T *)p.b, *C = (const T *)p.c;
    T *O = (T *)p.out;
    T ra[OUT ? kPerB : 1], rb[kPerB], rc[kPerC];
    auto row_of = [&](int64_t n) { return (rev ? t1 - 1 - n : t0 + n) * H + h; };   // n-th token's row
    auto load = [&](int64_t tb) {
#pragma unroll
        for (int k = 0; k < kPerB; ++k) {
            const int i = tid + k * kThreads;
            const int64_t n = tb + i / KD;
            const bool on = n < ntok;
            const int64_t at = on ? row_of(n) * KD + i % KD : 0;
            rb[k] = on ? B[at] : from_f32<T>(0.f);
            if (OUT) ra[k] = on ? A[at] : from_f32<T>(0.f);
        }
#pragma unroll
        for (int k = 0; k < kPerC; ++k) {
            const int i = tid + k * kThreads;
            const int64_t n = tb + i / kCols;
            rc[k] = n < ntok ? C[row_of(n) * vd + e0 + i % kCols] : from_f32<T>(0.f);
        }
    };
    load(0);
    __syncthreads();
    for (int64_t tb = 0; tb < ntok; tb += kTb) {
        const int nr = (int)min((int64_t)kTb, ntok - tb);
        if (tb && nb > 1) decay(step);
#pragma unroll
        for (int k = 0; k < kPerB; ++k) {
            const int i = tid + k * kThreads;
            bs[i / KD][i % KD] = to_f32(rb[k]);
            if (OUT) as[i / KD][i % KD] = to_f32(ra[k]) * (p.s_out * pw[i / KD][0]);
        }
#pragma unroll
        for (int k = 0; k < kPerC; ++k) {
            const int i = tid + k * kThreads;
            cs[i / kCols][i % kCols] = to_f32(rc[k]) * (p.s_upd * pw[i / kCols][1]);
        }
        __syncthreads();
        if (tb + kTb < ntok) load(tb + kTb);
        // kU tokens at a time: their sums over the lanes are independent of each other, and
        // the state's chain is one multiply-add per token
        auto tokens = [&](int r0, auto count) {
            constexpr int kU = decltype(count)::value;
            float o[kU][8];
#pragma unroll
            for (int q = 0; q < kU; ++q) {
                const int r = r0 + q;
                if (nb == 1 && tb + r) decay(step);
                float bv[4], cv[8], av[4];
                *(float4 *)&bv[0] = *(const float4 *)&bs[r][4 * dl];
                *(float4 *)&cv[0] = *(const float4 *)&cs[r][8 * eg];
                *(float4 *)&cv[4] = *(const float4 *)&cs[r][8 * eg + 4];
                if (OUT) *(float4 *)&av[0] = *(const float4 *)&as[r][4 * dl];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[q][j] = 0.f;
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        s[u][j] = fmaf(bv[u], cv[j], s[u][j]);
                        if (OUT) o[q][j] = fmaf(av[u], s[u][j], o[q][j]);
                    }
            }
            if (!OUT) return;
            // sum over the kLanes threads of the columns: each exchange halves the columns a
            // thread carries until it has one; lane bits give which
            int col = 0, lanes = kLanes;
#pragma unroll
            for (int n = 4; n; n >>= 1) {
                lanes >>= 1;
                const bool up = dl & lanes;
#pragma unroll
                for (int q = 0; q < kU; ++q)
#pragma unroll
                    for (int j = 0; j < n; ++j) {
                        const float send = up ? o[q][j] : o[q][j + n];
                        o[q][j] = (up ? o[q][j + n] : o[q][j]) + __shfl_xor_sync(kFull, send, lanes);
                    }
                if (up) col += n;
            }
#pragma unroll
            for (int q = 0; q < kU; ++q) {
#pragma unroll
                for (int n = kLanes / 16; n; n >>= 1) o[q][0] += __shfl_xor_sync(kFull, o[q][0], n);
                if (dl % (kLanes / 8) == 0) os[r0 + q][8 * eg + col] = o[q][0];
            }
        };
        int r = 0;
#pragma unroll 1
        for (; r + 2 <= nr; r += 2) tokens(r, std::integral_constant<int, 2>{});
        if (r < nr) tokens(r, std::integral_constant<int, 1>{});
        __syncthreads();
        if (OUT)
            for (int i = tid; i < nr * kCols; i += kThreads)
                O[row_of(tb + i / kCols) * vd + e0 + i % kCols] = from_f32<T>(os[i / kCols][i % kCols]);
    }
    float *to = decay_state_out(p, seg, H, h);
    if (!to) return;
    if (ntok > 0) decay(DecayFactor(gd * (float)((nb > 1 ? (ntok - 1) % kTb : 0) + (rev ? 1 : 0))));
    if (p.transposed) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *(float4 *)&to[(e0 + 8 * eg + j) * KD + 4 * dl] = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *(float4 *)&to[(4 * dl + u) * vd + e0 + 8 * eg + j] = *(const float4 *)&s[u][j];
    }
}

// A few tokens of every sequence, the state updated in place.  A block owns 64 columns of
// one (sequence, head)'s state: 256 threads hold kd / 16 rows x 4 columns each as float4,
// all loaded before anything else (32 KB a block in flight at kd = 128), so that the
// pass is bound by the state's traffic, 2 x 4 kd vd bytes.  The states go back with the
// evict-first policy: 256 sequences' of 16 heads are twice the L2, and plain stores push out
// lines that are still to be read (98.8 us against 80.8).  Sums over kd: a shuffle, then
// the 8 warps' partial sums through shared memory.  One token of 256 sequences, 16 heads x 128:
// 80.8 us, 6.7 TB/s, 98% of a copy's; of one sequence: 8 us, which is the launch and one chain of
// loads, sums and stores.
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
            for (int u = 0; u < kRows; ++u) __stcs(&S[(int64_t)4 * u * vd], s[u]);
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

// cur = s0; per segment in the order of the pass: cur = lam^len cur + its local sum (of its
// parts, in order), the state that enters the next segment, written over the sum.  A block
// takes 1024 elements of one (sequence, head).  Bound by the sums' latency, four on their way at a time: 18 boundaries
// of 16 heads x 128 x 128 12 us (one at a time 16.5; eight 12.3, and 14.5 against 12.4 where there
// are many short sequences), 16 with the slow heads' sums in three parts.
__global__ void __launch_bounds__(256)
decay_combine_kernel(const DecayGeom g, const __grid_constant__ Passes passes) {
    let_next_start();
    after_previous();
    const DecayPass &p = passes.p[blockIdx.y];
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
    const int sums = decay_parts(g, gd);
    const int64_t part_step = g.max_slots * g.H * st / 4;   // in float4
    float4 cur = p.s0 ? *(const float4 *)&p.s0[nh * st + at] : make_float4(0.f, 0.f, 0.f, 0.f);
    float *slots = p.slots + ((base - n) * g.H + h) * st + at;
    // (the stores would keep later loads behind them)
    constexpr int kAhead = 4;
    for (int64_t i0 = 0; i0 < cnt - 1; i0 += kAhead) {
        float4 x[kAhead];
        auto slot = [&](int64_t i) { return (float4 *)&slots[(p.rev ? cnt - 2 - i : i) * g.H * st]; };
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i0 + k < cnt - 1) x[k] = *slot(i0 + k);
        for (int j = 1; j < sums; ++j) {
            float4 y[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k < cnt - 1) y[k] = slot(i0 + k)[j * part_step];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k < cnt - 1)
                    x[k] = make_float4(x[k].x + y[k].x, x[k].y + y[k].y, x[k].z + y[k].z, x[k].w + y[k].w);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t i = i0 + k;
            if (i >= cnt - 1) break;
            // reversed: the last segment, which may be short, comes first
            const DecayFactor f = p.rev && i == 0 ? DecayFactor(gd * (float)(len - (cnt - 1) * g.seg_tokens)) : full;
            cur = make_float4(f(cur.x) + x[k].x, f(cur.y) + x[k].y, f(cur.z) + x[k].z, f(cur.w) + x[k].w);
            *slot(i) = cur;
        }
    }
}

Passes packed(const DecayPass *p, int n) {
    Passes a{};
    std::copy(p, p + n, a.p);
    return a;
}

// One launch per key width among the passes.
template <typename T, int KD>
cudaError_t rec_t(const DecayGeom &g, const DecayPass *p, int n, bool early, cudaStream_t stream) {
    DecayPass mine[kDecayMaxPasses];
    int k = 0, vd = 0;
    for (int i = 0; i < n; ++i)
        if (p[i].kd == KD) {
            mine[k++] = p[i];
            vd = std::max(vd, p[i].vd);
        }
    const int64_t blocks = g.max_segs * g.H * (vd / kCols);
    if (k == 0 || blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    ProfScope prof(stream, p[0].local ? "decay_rec_kernel (local)" : "decay_rec_kernel");
    auto kern = p[0].local ? decay_rec_kernel<T, KD, false> : decay_rec_kernel<T, KD, true>;
    const cudaError_t err = launch_early(early, kern, dim3((unsigned)blocks, (unsigned)k), 2 * KD, 0, stream, g,
                                         packed(mine, k));
    count_launch();
    return err;
}
template <typename T>
cudaError_t rec_all(const DecayGeom &g, const DecayPass *p, int n, bool early, cudaStream_t stream) {
    // a call's two launches are independent, but the next kernel waits for the second one only
    const bool both = std::any_of(p, p + n, [&](const DecayPass &q) { return q.kd != p[0].kd; });
    const cudaError_t err = rec_t<T, 128>(g, p, n, early, stream);
    return err == cudaSuccess ? rec_t<T, 64>(g, p, n, early && !both, stream) : err;
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

cudaError_t launch_decay_rec(const DecayGeom &g, const DecayPass *passes, int n, gdr_dtype_t dtype, bool early,
                             cudaStream_t stream) {
    if (n < 1 || n > kDecayMaxPasses) return cudaErrorInvalidValue;
    return dtype == GDR_BF16 ? rec_all<__nv_bfloat16>(g, passes, n, early, stream)
                             : rec_all<float>(g, passes, n, early, stream);
}

cudaError_t launch_decay_combine(const DecayGeom &g, const DecayPass *passes, int n, cudaStream_t stream) {
    const int64_t blocks = (int64_t)g.N * g.H * ((int64_t)passes[0].kd * passes[0].vd / 1024);
    if (blocks > 0x7fffffff || n < 1 || n > kDecayMaxPasses) return cudaErrorInvalidValue;
    ProfScope prof(stream, "decay_combine_kernel");
    const cudaError_t err = launch_early(true, decay_combine_kernel, dim3((unsigned)blocks, (unsigned)n), 256, 0,
                                         stream, g, packed(passes, n));
    count_launch();
    return err;
}

cudaError_t launch_decay_plan(const int32_t *cu_seqlens, const DecayGeom &g, int64_t *seq_start, int64_t *seg_base,
                              unsigned long long *next, int *status, cudaStream_t stream) {
    ProfScope prof(stream, "decay_plan_kernel");
    decay_plan_kernel<<<1, 1024, 0, stream>>>(cu_seqlens, g.N, g.T_total, g.seg_tokens, seq_start, seg_base, next,
                                              status);
    count_launch();
    return cudaGetLastError();
}

}  // namespace gdr
