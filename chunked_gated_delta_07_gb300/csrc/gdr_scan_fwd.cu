// gdr_scan_fwd.cu -- the gated scan forward over prompts, and token by token.
//
// Per (sequence, channel) h_t = alpha_t h_{t-1} + w(alpha_t) x_t (gdr_scan.cuh).  Two tensors are
// read and one is written, each once; a channel's step is a dozen operations and two to four
// special functions, so HBM bounds long calls as long as enough copies are under way.  A block's
// tile is 128 tokens x 32 channels: asynchronous copies bring the tiles ahead into shared memory
// while a lane keeps the decays and inputs of its run in registers, from the run's own pair to
// the second pass over it.
#include <algorithm>

#include "gdr_scan.cuh"

namespace gdr {
namespace {

using namespace scan;

constexpr int kL = 16;                           // tokens of a lane's run
constexpr int kWarps = kScanTile / (2 * kL);
constexpr int kThreads = 32 * kWarps;
template <typename T> constexpr int kBlocksPerSm = sizeof(T) == 2 ? 4 : 3;
template <typename T> constexpr int kDepth = sizeof(T) == 2 ? 3 : 2;   // tiles in shared memory
template <typename T> constexpr int kTileBytes = kWarps * 2 * kWarpTile<T, kL> * (int)sizeof(T);
template <typename T> constexpr int kSmem = kDepth<T> * kTileBytes<T>;

template <typename T, int GATE, int SRC>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<T>)
scan_fwd_kernel(const T *x, const T *a, const float *h0, T *out, float *hT, float *states, ScanShape s, int mode,
                int pairs, int *status) {
    constexpr bool kFine = sizeof(T) == 4;
    extern __shared__ uint4 ring_[];
    __shared__ __align__(16) float4 agg[2][kWarps][16];
    __shared__ __align__(16) float4 peer[2][kScanMaxCluster][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = lane >> 4, l = lane & 15;
    const int CS = s.cluster, rank = blockIdx.x % CS, unit = blockIdx.x / CS;
    const int c0 = unit % s.tiles * kScanChannels, c = c0 + 2 * l;
    const int first = unit / s.tiles * s.per_part, last = min(s.N, first + s.per_part);
    if (!offsets_ok(s)) {
        if (threadIdx.x == 0) set_status(status, GDR_ERR_BAD_SEQLENS);
        return;
    }
    const int p0 = seq_start(s, first), p1 = seq_start(s, last);
    const bool on0 = c < s.D, on1 = c + 1 < s.D;
    if (s.cu && hT && hT != h0 && c0 + lane < s.D)   // sequences of no tokens
        for (int n = first + warp + rank * kWarps; n < last; n += kWarps * CS)
            if (seq_start(s, n) == seq_start(s, n + 1))
                hT[(int64_t)n * s.D + c0 + lane] = h0 ? h0[(int64_t)n * s.D + c0 + lane] : 0.f;
    const int t0 = p0 / kScanTile, t1 = (p1 + kScanTile - 1) / kScanTile, steps = (t1 - t0 + CS - 1) / CS;
    const bool many = last - first > 1;
    T *ring = (T *)ring_ + warp * 2 * kWarpTile<T, kL>;
    constexpr int kSlot = kWarps * 2 * kWarpTile<T, kL>;
    const T *const src[2] = {x, a};
    auto ask = [&](int i, int slot) {
        const int64_t row = (int64_t)(t0 + i * (int64_t)CS + rank) * kScanTile + warp * 2 * kL;
        if (i < steps && row < p1)
            ask_tile<T, kL, 2>(ring + slot * kSlot, src, mode, (int)row, p0, p1, c0, s.D);
        copies_commit();
    };
    for (int i = 0; i < kDepth<T> - 1; ++i) ask(i, i);
    if (CS > 1) cluster_sync();   // every peer runs before its memory is written to
    Cursor cur{first, 0, -1};
    float carry0 = 0.f, carry1 = 0.f;
    int slot = 0;
    for (int i = 0; i < steps; ++i) {
        ask(i + kDepth<T> - 1, slot == 0 ? kDepth<T> - 1 : slot - 1);
        copies_wait<kDepth<T> - 1>();
        __syncwarp();
        const T *tile = ring + slot * kSlot;
        slot = slot == kDepth<T> - 1 ? 0 : slot + 1;
        const bool cuts = many || i == 0;
        const int64_t base = (int64_t)(t0 + i * (int64_t)CS + rank) * kScanTile;   // may lie behind the part
        const int p = (int)min(base + (warp * 2 + half) * kL, (int64_t)p1);
        const int lo = max(p, p0), hi = min(p + kL, p1);
        const bool whole = hi - lo == kL;
        const Marks m = marks_of(s, cur, first, last, p, lo, hi);
        float al[kL][2], u[kL][2], A0 = 1.f, A1 = 1.f, B0 = 0.f, B1 = 0.f;
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            const float2 xv = read2(tile, j, lane), av = read2(tile + kWarpTile<T, kL>, j, lane);
            const Gate g0 = gate_of<kFine, GATE, SRC, false>(av.x, s.b), g1 = gate_of<kFine, GATE, SRC, false>(av.y, s.b);
            al[j][0] = g0.alpha;
            al[j][1] = g1.alpha;
            u[j][0] = SRC == GDR_SOURCE_PLAIN ? xv.x : g0.w * xv.x;
            u[j][1] = SRC == GDR_SOURCE_PLAIN ? xv.y : g1.w * xv.y;
        }
        if (!whole) {
#pragma unroll
            for (int j = 0; j < kL; ++j)
                if (p + j < lo || p + j >= hi) {
                    al[j][0] = al[j][1] = 1.f;
                    u[j][0] = u[j][1] = 0.f;
                }
        }
        if (m.first) {
            int n = cur.n;
#pragma unroll
            for (int j = 0; j < kL; ++j)
                if (m.first >> j & 1) {
                    n = seq_from(s, n, p + j);
                    const float *h = h0 + (int64_t)n * s.D + c;
                    u[j][0] = fmaf(al[j][0], h0 && on0 ? h[0] : 0.f, u[j][0]);
                    u[j][1] = fmaf(al[j][1], h0 && on1 ? h[1] : 0.f, u[j][1]);
                    A0 = A1 = -1.f;
                    B0 = u[j][0];
                    B1 = u[j][1];
                } else {
                    B0 = fmaf(al[j][0], B0, u[j][0]);
                    B1 = fmaf(al[j][1], B1, u[j][1]);
                    decay_past_cut(A0, al[j][0]);
                    decay_past_cut(A1, al[j][1]);
                }
        } else {
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                B0 = fmaf(al[j][0], B0, u[j][0]);
                B1 = fmaf(al[j][1], B1, u[j][1]);
                A0 *= al[j][0];
                A1 *= al[j][1];
            }
        }
        // the first half's run, then both; the second half's lanes need the first's
        const float a0 = __shfl_xor_sync(kFull, A0, 16), a1 = __shfl_xor_sync(kFull, A1, 16);
        const float b0 = __shfl_xor_sync(kFull, B0, 16), b1 = __shfl_xor_sync(kFull, B1, 16);
        if (half == 0) {
            float wa0 = A0, wa1 = A1, wb0 = B0, wb1 = B1;
            follow(wa0, wb0, a0, b0, cuts);
            follow(wa1, wb1, a1, b1, cuts);
            agg[i & 1][warp][l] = make_float4(wa0, wa1, wb0, wb1);
        }
        __syncthreads();
        float h0v, h1v;
        if (CS == 1) {
            float e0 = carry0, e1 = carry1;
            h0v = e0;
            h1v = e1;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 r = agg[i & 1][w][l];
                if (w == warp) {
                    h0v = e0;
                    h1v = e1;
                }
                e0 = through(r.x, r.z, e0, cuts);
                e1 = through(r.y, r.w, e1, cuts);
            }
            carry0 = e0;
            carry1 = e1;
        } else {
            float pa0 = 1.f, pa1 = 1.f, pb0 = 0.f, pb1 = 0.f;   // of the warps in front; warp 0: of all
            const int upto = warp == 0 ? kWarps : warp;
            for (int w = 0; w < upto; ++w) {
                const float4 r = agg[i & 1][w][l];
                follow(pa0, pb0, r.x, r.z, cuts);
                follow(pa1, pb1, r.y, r.w, cuts);
            }
            if (warp == 0) {
                for (int r = half; r < CS; r += 2)
                    put_to_peer(&peer[i & 1][rank][l], r, make_float4(pa0, pa1, pb0, pb1));
                pa0 = pa1 = 1.f;
                pb0 = pb1 = 0.f;
            }
            cluster_sync();
            float e0 = carry0, e1 = carry1;
            h0v = e0;
            h1v = e1;
            for (int r = 0; r < CS; ++r) {
                const float4 v = peer[i & 1][r][l];
                if (r == rank) {
                    h0v = e0;
                    h1v = e1;
                }
                e0 = through(v.x, v.z, e0, cuts);
                e1 = through(v.y, v.w, e1, cuts);
            }
            carry0 = e0;
            carry1 = e1;
            h0v = through(pa0, pb0, h0v, cuts);
            h1v = through(pa1, pb1, h1v, cuts);
        }
        if (half) {
            h0v = through(a0, b0, h0v, cuts);
            h1v = through(a1, b1, h1v, cuts);
        }
        if (whole && on1 && pairs && !(m.first | m.last)) {
            if (out) {
                T *o = out + (int64_t)p * s.D + c;
#pragma unroll
                for (int j = 0; j < kL; ++j) {
                    h0v = fmaf(al[j][0], h0v, u[j][0]);
                    h1v = fmaf(al[j][1], h1v, u[j][1]);
                    write2(o, h0v, h1v);
                    o += s.D;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kL; ++j) {
                    h0v = fmaf(al[j][0], h0v, u[j][0]);
                    h1v = fmaf(al[j][1], h1v, u[j][1]);
                }
            }
        } else if (on0) {
            int n = cur.n;
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const bool cut = m.first >> j & 1;
                h0v = fmaf(al[j][0], cut ? 0.f : h0v, u[j][0]);
                h1v = fmaf(al[j][1], cut ? 0.f : h1v, u[j][1]);
                if (cut) {   // as the sum above has it, whatever alpha is
                    h0v = u[j][0];
                    h1v = u[j][1];
                }
                const int t = p + j;
                if (t < lo || t >= hi) continue;
                if (out) {
                    T *o = out + (int64_t)t * s.D + c;
                    o[0] = from_f32<T>(h0v);
                    if (on1) o[1] = from_f32<T>(h1v);
                }
                if (hT && (m.last >> j & 1)) {
                    n = seq_from(s, n, t);
                    hT[(int64_t)n * s.D + c] = h0v;
                    if (on1) hT[(int64_t)n * s.D + c + 1] = h1v;
                }
            }
        }
        // the state behind a tile's last token
        if (states && half == 1 && warp == kWarps - 1 && p + kL == hi && base + kScanTile == hi) {
            float *d = states + (int64_t)(base / kScanTile) * s.D + c;
            if (on0) d[0] = h0v;
            if (on1) d[1] = h1v;
        }
    }
    copies_wait<0>();
}

template <typename T, int GATE, int SRC>
cudaError_t launch_fwd_t(const ScanFwd &t, ScanShape s, int sms, int *status, cudaStream_t stream) {
    auto kern = scan_fwd_kernel<T, GATE, SRC>;
    scan_divide(s, (int64_t)sms * kBlocksPerSm<T>);
    const bool wide = s.D % wide_elems<T>() == 0 && ((uintptr_t)t.x | (uintptr_t)t.a) % 16 == 0;
    const bool even = s.D % 2 == 0;
    const bool pair = sizeof(T) == 4 || (even && ((uintptr_t)t.x | (uintptr_t)t.a) % 4 == 0);
    const int mode = wide ? kWide : pair ? kPair : kSingle;
    const int pairs = even && (uintptr_t)t.out % (2 * sizeof(T)) == 0;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<T>);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)s.tiles * s.parts * s.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem<T>;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)s.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = s.cluster > 1 ? 1 : 0;
    ProfScope prof(stream, "scan_fwd_kernel");
    err = cudaLaunchKernelEx(&cfg, kern, (const T *)t.x, (const T *)t.a, t.h0, (T *)t.out, t.hT, t.states, s, mode, pairs,
                             status);
    count_launch();
    return err;
}

// One (sequence, channel) to a thread, the next token's inputs on their way while a token is
// computed.  Bound by the launch for a few sequences, by HBM beyond: the states, then the tokens.
template <typename T, int GATE, int SRC>
__global__ void __launch_bounds__(256)
scan_step_kernel(const T *__restrict__ x, const T *__restrict__ a, float *__restrict__ state, T *__restrict__ out,
                 int64_t units, int T_, int D, float b) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= units) return;
    const int64_t n = i / D, at = n * T_ * D + (i - n * D);
    float h = state[i];
    T xv = x[at], av = a[at];
    for (int t = 0; t < T_; ++t) {
        const int64_t next = at + (int64_t)(t + 1 < T_ ? t + 1 : t) * D;
        const T xn = x[next], an = a[next];
        const Gate g = gate_of<sizeof(T) == 4, GATE, SRC, false>(to_f32(av), b);
        h = fmaf(g.alpha, h, g.w * to_f32(xv));
        out[at + (int64_t)t * D] = from_f32<T>(h);
        xv = xn;
        av = an;
    }
    state[i] = h;
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanFwd &t, ScanShape s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                            int sms, int *status, cudaStream_t stream) {
    return with_form(gate, source, [&](auto g, auto w) {
        return dtype == GDR_BF16 ? launch_fwd_t<__nv_bfloat16, g(), w()>(t, s, sms, status, stream)
                                 : launch_fwd_t<float, g(), w()>(t, s, sms, status, stream);
    });
}

cudaError_t launch_scan_step(const void *x, const void *a, float *state, void *out, int N, int T, int D, float b,
                             gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source, cudaStream_t stream) {
    return with_form(gate, source, [&](auto g, auto w) {
        const int64_t units = (int64_t)N * D;
        const unsigned grid = (unsigned)((units + 255) / 256);
        ProfScope prof(stream, "scan_step_kernel");
        if (dtype == GDR_BF16)
            scan_step_kernel<__nv_bfloat16, g(), w()><<<grid, 256, 0, stream>>>(
                (const __nv_bfloat16 *)x, (const __nv_bfloat16 *)a, state, (__nv_bfloat16 *)out, units, T, D, b);
        else
            scan_step_kernel<float, g(), w()><<<grid, 256, 0, stream>>>((const float *)x, (const float *)a, state,
                                                                        (float *)out, units, T, D, b);
        count_launch();
        return cudaGetLastError();
    });
}

}  // namespace gdr
