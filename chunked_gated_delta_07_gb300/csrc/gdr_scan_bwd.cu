// gdr_scan_bwd.cu -- gradients of the gated scan.
//
// With l_t the gradient of h_t and r_t that of h_{t-1} through alpha_t:
//     l_t = dout_t + r_{t+1} (the last token's holds dhT too),   r_t = alpha_t l_t,  dh0 = r_1
//     dx_t = w l_t,   da_t = l_t (alpha_t h_{t-1} + w'(g_t) x_t) g'(a_t)
// One pass over the tiles from the last to the first: the gradient is chained backwards as the
// forward pass chains its states (gdr_scan.cuh), and the states within a tile are chained
// forwards again from the one that the forward pass kept in front of it.  Three tensors are
// read and two written, each once.  The pairs of both directions share their A.
#include <algorithm>

#include "gdr_scan.cuh"

namespace gdr {
namespace {

using namespace scan;

constexpr int kL = 8;
constexpr int kWarps = kScanTile / (2 * kL);
constexpr int kThreads = 32 * kWarps;
constexpr int kBlocksPerSm = 2;
template <typename T> constexpr int kDepth = sizeof(T) == 2 ? 4 : 2;
template <typename T> constexpr int kTileBytes = kWarps * 3 * kWarpTile<T, kL> * (int)sizeof(T);
template <typename T> constexpr int kSmem = kDepth<T> * kTileBytes<T>;

template <typename T, int GATE, int SRC>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
scan_bwd_kernel(const T *x, const T *a, const T *dout, const float *__restrict__ h0, const float *__restrict__ dhT,
                const float *__restrict__ states, T *dx, T *da, float *dh0, ScanShape s, int mode, int pairs, int *status) {
    constexpr bool kFine = sizeof(T) == 4;
    extern __shared__ uint4 ring_[];
    __shared__ __align__(16) float4 agg[2][kWarps][16];    // A, and the gradient's B
    __shared__ __align__(16) float2 aggh[2][kWarps][16];   // the state's B
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
    if (s.cu && dh0 && c0 + lane < s.D)   // sequences of no tokens
        for (int n = first + warp + rank * kWarps; n < last; n += kWarps * CS)
            if (seq_start(s, n) == seq_start(s, n + 1))
                dh0[(int64_t)n * s.D + c0 + lane] = dhT ? dhT[(int64_t)n * s.D + c0 + lane] : 0.f;
    const int t0 = p0 / kScanTile, t1 = (p1 + kScanTile - 1) / kScanTile, steps = (t1 - t0 + CS - 1) / CS;
    const bool many = last - first > 1;
    T *ring = (T *)ring_ + warp * 3 * kWarpTile<T, kL>;
    constexpr int kSlot = kWarps * 3 * kWarpTile<T, kL>;
    const T *const src[3] = {x, a, dout};
    // step i of this block: tile t1 - 1 - (i CS + rank), none below t0
    auto tile_of = [&](int i) { return (int64_t)t1 - 1 - (i * (int64_t)CS + rank); };
    auto ask = [&](int i, int slot) {
        const int64_t t = tile_of(i);
        if (i < steps && t >= t0)
            ask_tile<T, kL, 3>(ring + slot * kSlot, src, mode, (int)(t * kScanTile) + warp * 2 * kL, p0, p1, c0, s.D);
        copies_commit();
    };
    for (int i = 0; i < kDepth<T> - 1; ++i) ask(i, i);
    if (CS > 1) cluster_sync();
    Cursor cur{first, 0, -1};
    float carry0 = 0.f, carry1 = 0.f;
    int slot = 0;
    for (int i = 0; i < steps; ++i) {
        ask(i + kDepth<T> - 1, slot == 0 ? kDepth<T> - 1 : slot - 1);
        const int64_t tile_no = tile_of(i);
        const bool there = tile_no >= t0;
        const bool cuts = many || i == steps - 1;
        // the state in front of the tile: kept by the forward pass behind the tile before
        float s0 = 0.f, s1 = 0.f;
        if (there && tile_no * kScanTile > p0) {
            const float *st = states + (tile_no - 1) * s.D + c;
            if (on0) s0 = st[0];
            if (on1) s1 = st[1];
        }
        copies_wait<kDepth<T> - 1>();
        __syncwarp();
        const T *tile = ring + slot * kSlot;
        slot = slot == kDepth<T> - 1 ? 0 : slot + 1;
        const int p = there ? (int)(tile_no * kScanTile) + (warp * 2 + half) * kL : p0 - kL;
        const int lo = max(p, p0), hi = min(p + kL, p1);
        const bool whole = hi - lo == kL;
        const Marks m = marks_of(s, cur, first, last, p, lo, hi);
        float al[kL][2], w[kL][2], qs[kL][2], qd[kL][2];
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            const float2 xv = read2(tile, j, lane), av = read2(tile + kWarpTile<T, kL>, j, lane);
            const Gate g0 = gate_of<kFine, GATE, SRC, true>(av.x, s.b), g1 = gate_of<kFine, GATE, SRC, true>(av.y, s.b);
            al[j][0] = g0.alpha;
            al[j][1] = g1.alpha;
            w[j][0] = g0.w;
            w[j][1] = g1.w;
            qs[j][0] = g0.slope * g0.alpha;
            qs[j][1] = g1.slope * g1.alpha;
            qd[j][0] = g0.dw * xv.x;
            qd[j][1] = g1.dw * xv.y;
        }
        if (!whole) {
#pragma unroll
            for (int j = 0; j < kL; ++j)
                if (p + j < lo || p + j >= hi) {
                    al[j][0] = al[j][1] = 1.f;
                    w[j][0] = w[j][1] = 0.f;
                }
        }
        // a token's input and gradient; zeros outside the part (whose place in shared memory may
        // never have been filled)
        auto x_at = [&](int j) { return whole || (p + j >= lo && p + j < hi) ? read2(tile, j, lane) : make_float2(0.f, 0.f); };
        auto d_at = [&](int j) {
            return whole || (p + j >= lo && p + j < hi) ? read2(tile + 2 * kWarpTile<T, kL>, j, lane) : make_float2(0.f, 0.f);
        };
        float A0 = 1.f, A1 = 1.f, B0 = 0.f, B1 = 0.f, R0 = 0.f, R1 = 0.f;
        const bool marked = m.first | m.last;
        if (marked) {
            int n = cur.n;
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const float2 xv = x_at(j);
                if (m.first >> j & 1) {
                    n = seq_from(s, n, p + j);
                    const float *h = h0 + (int64_t)n * s.D + c;
                    B0 = h0 && on0 ? h[0] : 0.f;
                    B1 = h0 && on1 ? h[1] : 0.f;
                    A0 = A1 = -1.f;
                }
                B0 = fmaf(al[j][0], B0, w[j][0] * xv.x);
                B1 = fmaf(al[j][1], B1, w[j][1] * xv.y);
                decay_past_cut(A0, al[j][0]);
                decay_past_cut(A1, al[j][1]);
            }
            // n: the sequence of the run's last token
            n = hi > lo ? seq_from(s, n, hi - 1) : n;
#pragma unroll
            for (int j = kL - 1; j >= 0; --j) {
                float2 d = d_at(j);
                if (m.last >> j & 1) {
                    while (seq_start(s, n) > p + j) --n;
                    if (dhT) {
                        const float *e = dhT + (int64_t)n * s.D + c;
                        d.x += on0 ? e[0] : 0.f;
                        d.y += on1 ? e[1] : 0.f;
                    }
                }
                R0 = al[j][0] * (d.x + R0);
                R1 = al[j][1] * (d.y + R1);
                if (m.first >> j & 1) R0 = R1 = 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const float2 xv = x_at(j);
                B0 = fmaf(al[j][0], B0, w[j][0] * xv.x);
                B1 = fmaf(al[j][1], B1, w[j][1] * xv.y);
                A0 *= al[j][0];
                A1 *= al[j][1];
            }
#pragma unroll
            for (int j = kL - 1; j >= 0; --j) {
                const float2 d = d_at(j);
                R0 = al[j][0] * (d.x + R0);
                R1 = al[j][1] * (d.y + R1);
            }
        }
        // the other half's run
        const float oa0 = __shfl_xor_sync(kFull, A0, 16), oa1 = __shfl_xor_sync(kFull, A1, 16);
        const float ob0 = __shfl_xor_sync(kFull, B0, 16), ob1 = __shfl_xor_sync(kFull, B1, 16);
        const float or0 = __shfl_xor_sync(kFull, R0, 16), or1 = __shfl_xor_sync(kFull, R1, 16);
        if (half == 0) {   // states: this run, then the other; gradients: the other, then this one
            float f0 = B0, f1 = B1, g0 = or0, g1 = or1, fa0 = A0, fa1 = A1, ga0 = oa0, ga1 = oa1;
            follow(fa0, f0, oa0, ob0, cuts);
            follow(fa1, f1, oa1, ob1, cuts);
            follow(ga0, g0, A0, R0, cuts);
            follow(ga1, g1, A1, R1, cuts);
            // a cut in either run shows in both products' signs
            agg[i & 1][warp][l] = make_float4(fa0, fa1, g0, g1);
            aggh[i & 1][warp][l] = make_float2(f0, f1);
        }
        __syncthreads();
        // the state that enters the run
        float h0v = s0, h1v = s1;
        for (int v = 0; v < warp; ++v) {
            const float4 r = agg[i & 1][v][l];
            const float2 b = aggh[i & 1][v][l];
            h0v = through(r.x, b.x, h0v, cuts);
            h1v = through(r.y, b.y, h1v, cuts);
        }
        if (half) {
            h0v = through(oa0, ob0, h0v, cuts);
            h1v = through(oa1, ob1, h1v, cuts);
        }
        // the gradient that enters it
        float r0, r1;
        {
            if (CS == 1) {
                float e0 = carry0, e1 = carry1;
                r0 = e0;
                r1 = e1;
#pragma unroll
                for (int v = kWarps - 1; v >= 0; --v) {
                    const float4 r = agg[i & 1][v][l];
                    if (v == warp) {
                        r0 = e0;
                        r1 = e1;
                    }
                    e0 = through(r.x, r.z, e0, cuts);
                    e1 = through(r.y, r.w, e1, cuts);
                }
                carry0 = e0;
                carry1 = e1;
            } else {
                float pa0 = 1.f, pa1 = 1.f, pb0 = 0.f, pb1 = 0.f;   // of the warps behind
                for (int v = kWarps - 1; v > warp; --v) {
                    const float4 r = agg[i & 1][v][l];
                    follow(pa0, pb0, r.x, r.z, cuts);
                    follow(pa1, pb1, r.y, r.w, cuts);
                }
                if (warp == 0) {   // and the tile's
                    const float4 r = agg[i & 1][0][l];
                    float wa0 = pa0, wa1 = pa1, wb0 = pb0, wb1 = pb1;
                    follow(wa0, wb0, r.x, r.z, cuts);
                    follow(wa1, wb1, r.y, r.w, cuts);
                    for (int k = half; k < CS; k += 2) put_to_peer(&peer[i & 1][rank][l], k, make_float4(wa0, wa1, wb0, wb1));
                }
                cluster_sync();
                float e0 = carry0, e1 = carry1;
                r0 = e0;
                r1 = e1;
                for (int k = 0; k < CS; ++k) {
                    const float4 v = peer[i & 1][k][l];
                    if (k == rank) {
                        r0 = e0;
                        r1 = e1;
                    }
                    e0 = through(v.x, v.z, e0, cuts);
                    e1 = through(v.y, v.w, e1, cuts);
                }
                carry0 = e0;
                carry1 = e1;
                r0 = through(pa0, pb0, r0, cuts);
                r1 = through(pa1, pb1, r1, cuts);
            }
        }
        if (!half) {
            r0 = through(oa0, or0, r0, cuts);
            r1 = through(oa1, or1, r1, cuts);
        }
        // forwards: qs := (alpha h_{t-1} + w' x) g'
        if (m.first) {
            int n = cur.n;
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const float2 xv = x_at(j);
                if (m.first >> j & 1) {
                    n = seq_from(s, n, p + j);
                    const float *h = h0 + (int64_t)n * s.D + c;
                    h0v = h0 && on0 ? h[0] : 0.f;
                    h1v = h0 && on1 ? h[1] : 0.f;
                }
                qs[j][0] = fmaf(qs[j][0], h0v, qd[j][0]);
                qs[j][1] = fmaf(qs[j][1], h1v, qd[j][1]);
                h0v = fmaf(al[j][0], h0v, w[j][0] * xv.x);
                h1v = fmaf(al[j][1], h1v, w[j][1] * xv.y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const float2 xv = x_at(j);
                qs[j][0] = fmaf(qs[j][0], h0v, qd[j][0]);
                qs[j][1] = fmaf(qs[j][1], h1v, qd[j][1]);
                h0v = fmaf(al[j][0], h0v, w[j][0] * xv.x);
                h1v = fmaf(al[j][1], h1v, w[j][1] * xv.y);
            }
        }
        // backwards
        if (whole && on1 && pairs && !marked) {
            const int64_t off = (int64_t)(p + kL - 1) * s.D + c;
            T *ox = dx + off, *oa = da + off;
#pragma unroll
            for (int j = kL - 1; j >= 0; --j) {
                const float2 d = d_at(j);
                const float l0 = d.x + r0, l1 = d.y + r1;
                write2(ox, w[j][0] * l0, w[j][1] * l1);
                write2(oa, l0 * qs[j][0], l1 * qs[j][1]);
                r0 = al[j][0] * l0;
                r1 = al[j][1] * l1;
                ox -= s.D;
                oa -= s.D;
            }
        } else if (on0 && hi > lo) {
            int n = seq_from(s, cur.n, hi - 1);
#pragma unroll
            for (int j = kL - 1; j >= 0; --j) {
                const int t = p + j;
                if (t < lo || t >= hi) continue;   // nothing there: alpha = 1
                float2 d = d_at(j);
                if (m.last >> j & 1) {
                    // nothing comes from behind a sequence's end
                    while (seq_start(s, n) > t) --n;
                    r0 = r1 = 0.f;
                    if (dhT) {
                        const float *e = dhT + (int64_t)n * s.D + c;
                        d.x += e[0];
                        d.y += on1 ? e[1] : 0.f;
                    }
                }
                const float l0 = d.x + r0, l1 = d.y + r1;
                T *ox = dx + (int64_t)t * s.D + c, *oa = da + (int64_t)t * s.D + c;
                ox[0] = from_f32<T>(w[j][0] * l0);
                oa[0] = from_f32<T>(l0 * qs[j][0]);
                if (on1) {
                    ox[1] = from_f32<T>(w[j][1] * l1);
                    oa[1] = from_f32<T>(l1 * qs[j][1]);
                }
                r0 = al[j][0] * l0;
                r1 = al[j][1] * l1;
                if (dh0 && (m.first >> j & 1)) {
                    float *e = dh0 + (int64_t)n * s.D + c;
                    e[0] = r0;
                    if (on1) e[1] = r1;
                }
            }
        }
    }
    copies_wait<0>();
}

template <typename T, int GATE, int SRC>
cudaError_t launch_bwd_t(const ScanBwd &t, ScanShape s, int sms, int *status, cudaStream_t stream) {
    auto kern = scan_bwd_kernel<T, GATE, SRC>;
    scan_divide(s, (int64_t)sms * kBlocksPerSm);
    const uintptr_t ins = (uintptr_t)t.x | (uintptr_t)t.a | (uintptr_t)t.dout, outs = (uintptr_t)t.dx | (uintptr_t)t.da;
    const bool wide = s.D % wide_elems<T>() == 0 && ins % 16 == 0, even = s.D % 2 == 0;
    const int mode = wide ? kWide : sizeof(T) == 4 || (even && ins % 4 == 0) ? kPair : kSingle;
    const int pairs = even && outs % (2 * sizeof(T)) == 0;
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
    ProfScope prof(stream, "scan_bwd_kernel");
    err = cudaLaunchKernelEx(&cfg, kern, (const T *)t.x, (const T *)t.a, (const T *)t.dout, t.h0, t.dhT, t.states,
                             (T *)t.dx, (T *)t.da, t.dh0, s, mode, pairs, status);
    count_launch();
    return err;
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanBwd &t, ScanShape s, gdr_dtype_t dtype, gdr_gate_t gate, gdr_source_t source,
                            int sms, int *status, cudaStream_t stream) {
    return with_form(gate, source, [&](auto g, auto w) {
        return dtype == GDR_BF16 ? launch_bwd_t<__nv_bfloat16, g(), w()>(t, s, sms, status, stream)
                                 : launch_bwd_t<float, g(), w()>(t, s, sms, status, stream);
    });
}

}  // namespace gdr
