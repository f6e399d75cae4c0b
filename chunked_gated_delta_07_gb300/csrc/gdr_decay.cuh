// gdr_decay.cuh -- linear attention with one constant decay per head: what its kernel
// families share.
//
// Forward and backward are the same map.  With lam = exp(log_decay[h]) a pass takes token
// rows A, B (width kd) and C (width vd) and computes, per (sequence, head),
//     S_t = lam S_{t-1} + s_upd b_t c_t^T,   out_t = s_out S_t^T a_t             (forward)
//     R_t = E_{t+1} + s_upd b_t c_t^T,  E_t = lam R_t,  out_t = s_out R_t^T a_t  (reversed)
// so that with o = scale S^T q the calls are
//     out, hT : forward   (A, B, C) = (q, k, v),     s_upd = 1,     s_out = scale
//     dq      : forward   (dout, v, k), state H^T,   s_upd = 1,     s_out = scale
//     dk      : reversed  (v, dout, q), state dH^T,  s_upd = scale, s_out = 1
//     dv, dh0 : reversed  (k, q, dout), state dH,    s_upd = scale, s_out = 1
// where the reversed state enters as dhT at the last token and leaves as dh0.
//
// A long sequence is cut into segments of seg_tiles tiles.  A local pass sums each
// segment's own writes, decayed to its end (its start, reversed), combine chains the sums
// into the states that cross the segments' boundaries, and the output pass runs every
// segment from its entering state.  On the tensor cores the local pass skips the tokens that
// the decay leaves nothing of.  It does leave a NaN of a NaN or an infinity; the output pass
// reads all tokens, and where its outputs show such a value, a launch behind it runs the
// sequence's head again, uncut.  Boundary b of sequence n lies between its segments b and
// b + 1 and has the slot seg_base[n] - n + b.
#pragma once

#include "gdr_internal.cuh"

namespace gdr {

constexpr int kDecayTile = 128;   // tokens per tile

struct DecayGeom {
    Plan p;                  // packed input only (no tiles)
    bool dense;
    int N, H;
    int64_t T_per, T_total;  // tokens per sequence (dense) / over all sequences
    int64_t seg_tokens;      // tokens per segment (tensor cores: a multiple of kDecayTile)
    int64_t segs_per_seq;    // dense: segments of a sequence
    int64_t max_segs;        // upper bound on the segments of all sequences
    int64_t max_slots;       // upper bound on the segment boundaries inside sequences
    int parts;               // pieces that a local pass cuts a segment into at most ...
    int64_t part_tokens;     // ... of this many tokens each, counted from where its sum ends
    const float *log_decay;  // [H]
};

struct DecayPass {
    const void *a, *b, *c;   // [rows][H][kd], [rows][H][kd], [rows][H][vd]
    void *out;               // [rows][H][vd]
    const float *s0;         // entering states [N][H][...] or null (zero)
    float *sT;               // leaving states [N][H][...] or null
    float *slots;            // boundary states [max_slots][H][...] or null (no segments); as
                             // many again for the sums of each further part
    int kd, vd;
    // the states in memory are [kd][vd], or [vd][kd] (the pass's state transposed)
    bool transposed;
    bool rev;
    bool local;              // sum each segment's own writes into slots; no outputs
    float s_upd, s_out;
};

// One segment: sequence n, tokens [t0, t1) of the packed axis.
struct DecaySeg {
    int n;
    int64_t t0, t1, slot;    // slot of the boundary after the segment (before it: slot - 1)
    bool first, last;        // within the sequence
};

#ifdef __CUDACC__
__device__ __forceinline__ bool decay_segment(const DecayGeom &g, int64_t s, DecaySeg &o) {
    int64_t i, cnt, base, beg, end;
    if (g.dense) {
        o.n = (int)(s / g.segs_per_seq);
        if (o.n >= g.N) return false;
        base = o.n * g.segs_per_seq;
        cnt = g.segs_per_seq;
        beg = o.n * g.T_per;
        end = beg + g.T_per;
    } else {
        o.n = find_owner(g.p.seg_base, g.N, s);
        if (o.n < 0) return false;
        base = g.p.seg_base[o.n];
        cnt = g.p.seg_base[o.n + 1] - base;
        beg = g.p.seq_start[o.n];
        end = g.p.seq_start[o.n + 1];
    }
    i = s - base;
    o.t0 = min(end, beg + i * g.seg_tokens);
    o.t1 = min(end, o.t0 + g.seg_tokens);
    o.slot = base - o.n + i;
    o.first = i == 0;
    o.last = i == cnt - 1;
    return true;
}

// Natural log-decay of a head; -inf (a head that keeps nothing) becomes a finite value
// with the same powers, so that 0 steps still give exp(0) = 1.
__device__ __forceinline__ float decay_log(const float *log_decay, int h) {
    const float g = log_decay[h];
    return g < -1e30f ? -1e30f : g;
}

// x exp(n g), for few or many elements x with one n g.  Near 1 the factor goes in as
// x + x (e^{ng} - 1): e^{ng} itself rounds to 24 bits, and a state that is decayed again and
// again takes that error each time in the same direction.  Further from 1 the difference
// would cancel, and few factors reach far.
struct DecayFactor {
    float f;
    bool near1;
    __device__ __forceinline__ explicit DecayFactor(float ng) : near1(ng > -0.5f) {
        f = near1 ? expm1f(ng) : expf(ng);
    }
    __device__ __forceinline__ float operator()(float x) const { return fmaf(x, f, near1 ? x : 0.f); }
};

// Tokens after which exp(n g) is below fp32's smallest normal number, e^-87.3: what a local
// pass on the tensor cores need not read.
__device__ __forceinline__ int64_t decay_reach(float g, int64_t n) {
    if (!(g < 0.f)) return n;
    const float r = 88.f / -g;
    return r < (float)n ? min(n, (int64_t)r + 1) : n;
}

// Parts of a segment that the local pass sums for a head with log-decay g, and combine adds.
__device__ __forceinline__ int decay_parts(const DecayGeom &geom, float g) {
    const int64_t reach = decay_reach(g, geom.seg_tokens);
    return (int)min((int64_t)geom.parts, (reach + geom.part_tokens - 1) / geom.part_tokens);
}

// Where a pass's segment finds its entering state and leaves its last one (null: zero, or
// not wanted), given the offset of (head, state) inside one slot or sequence.
__device__ __forceinline__ const float *decay_state_in(const DecayPass &p, const DecaySeg &s, int H, int h) {
    const int64_t st = (int64_t)p.kd * p.vd;
    if (p.local) return nullptr;   // starts from zero
    if (p.rev ? s.last : s.first) return p.s0 ? p.s0 + ((int64_t)s.n * H + h) * st : nullptr;
    return p.slots + ((p.rev ? s.slot : s.slot - 1) * H + h) * st;
}
__device__ __forceinline__ float *decay_state_out(const DecayPass &p, const DecaySeg &s, int H, int h) {
    const int64_t st = (int64_t)p.kd * p.vd;
    if (p.local) return p.slots + ((p.rev ? s.slot - 1 : s.slot) * H + h) * st;
    if (p.rev ? s.first : s.last) return p.sT ? p.sT + ((int64_t)s.n * H + h) * st : nullptr;
    return nullptr;
}
#endif

constexpr int kDecayMaxPasses = 3;

// The plan of packed input: seq_start and seg_base of g.p (N + 1 each) from the offsets,
// which it validates, and the two unit counters zeroed (gdr_decay.cu).
cudaError_t launch_decay_plan(const int32_t *cu_seqlens, const DecayGeom &g, int64_t *seq_start, int64_t *seg_base,
                              unsigned long long *next, int *status, cudaStream_t stream);
// Token by token on the CUDA cores (gdr_decay.cu): any dtype, kd and vd in {64, 128}; n
// independent passes, all local or all not.  `early`: the kernel before it in the stream is
// the same call's.
cudaError_t launch_decay_rec(const DecayGeom &g, const DecayPass *passes, int n, gdr_dtype_t dtype, bool early,
                             cudaStream_t stream);
// T tokens of N sequences, the state [N, H, dk, dv] updated in place (gdr_decay.cu).
cudaError_t launch_decay_step(const void *q, const void *k, const void *v, const float *log_decay, float *state,
                              void *out, gdr_dtype_t dtype, int N, int64_t T, int H, int dk, int dv, float scale,
                              cudaStream_t stream);
// On the tensor cores (gdr_decay_tc.cu): bf16, token tensors 16-byte aligned, fewer than
// 2^31 - 128 token rows.  Passes of one launch are independent and all local or all not.
// `next`: a zeroed counter that hands out the units, or null (few units of equal length).
// `again`: runs, uncut, every (sequence, head, pass) of cut sequences whose outputs, by the launch
// before, show a value that is not finite and that a local sum may have skipped.
cudaError_t launch_decay_tc(const DecayGeom &g, const DecayPass *passes, int n, int sms, unsigned long long *next,
                            bool early, int *status, cudaStream_t stream, bool again = false);
// Chains the local sums in `slots` of n passes into boundary states, from s0 (null: zero).
cudaError_t launch_decay_combine(const DecayGeom &g, const DecayPass *passes, int n, cudaStream_t stream);

}  // namespace gdr
