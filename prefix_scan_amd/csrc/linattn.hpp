// linattn.hpp -- what the linear-attention kernels and their host code share.
//
// Linear attention with a decay is a prefix scan whose elements are pairs
// (decay, matrix) under (l, S) o (r, U) = (l r, r S + U).  Every product the
// operator and its gradient need is one "sweep" over the tokens of a
// sequence, in their order or in reverse:
//
//   out(i) = out_scale * ( sum_{j <= i} p^(i-j) pair_scale (a_i . b_j) c_j
//                          + p^(i+1-shift) Z0^T a_i )            p = e^g
//   Zend   = p^len Z0 + sum_j p^(len-1+shift-j) pair_scale b_j c_j^T
//
// with a, b of width m, c and out of width n and Z an m x n state:
//   forward    a, b, c = q, k, v     order forward,  shift 0
//   dq         a, b, c = do, v, k    order forward,  shift 0, Z transposed
//   dk         a, b, c = v, do, q    order reversed, shift 1, Z transposed
//   dv         a, b, c = k, q, do    order reversed, shift 1
// (dk(t) = R(t) v(t), dv(t) = R(t)^T k(t) with R the decayed sum of
// scale q do^T over the later tokens, to which the gradient of the final
// state enters undecayed at the last token: shift 1.)
//
// A sequence is cut into segments of seg_len tokens, one workgroup each, so
// that few long sequences still fill the GPU: a first kernel sums every
// segment's own contribution to the state (but the last's, which none reads),
// a second scans those sums along the sequence, and the third sweeps each
// segment from its entering state.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace libscan {

constexpr int kMaxSweeps = 3;
constexpr int kLinattnWidth = 128;      // largest m and n
// A segment of a sequence of no more than these adds up the states of those
// before it by itself: cheaper than the scan's own launch and second pass.
constexpr uint64_t kFewSegments = 4;

// Rows of one tensor: token t of sequence s, head h starts at element
// s * seq + t * tok + (h / share) * head.
struct Rows {
    const void *p;
    int64_t seq, tok, head;
    uint32_t share;
};

struct Sweep {
    Rows a, b, c;
    void *out;
    int64_t out_seq, out_tok, out_head;
    int m, n;
    int rev, shift;
    int out_f32;                 // out holds floats (partial gradients of shared heads)
    int out_whole;               // its rows start on 16 bytes and are whole multiples of them
    float pair_scale, out_scale;
    const float *state_in;       // per (sequence, head) m * n floats, or null
    float *state_out;
    int64_t state_m, state_n;    // element strides of a state's two axes
};

struct SweepSet {
    Sweep s[kMaxSweeps];
    int count;
    int dtype;                   // LIBSCAN_F32 / BF16 / F16
    const float *log_decay;      // [heads]
    const uint32_t *ends;        // inclusive run ends, or null: `tokens` per sequence
    uint32_t seqs, heads;
    uint64_t tokens;             // of each sequence, or in all when ends is given
    uint64_t seg_len;            // 0: sequences are not cut
    uint32_t items;              // workgroups along the tokens
    uint32_t slots;              // states of segments, of each head and sweep
    float *seg;                  // [sweeps][slots][heads] of them
    bool aligned;                // every row starts on 16 bytes and is a whole number of them
    const uint32_t *clear_from;  // outputs are zeroed from this token on, or null
};

// Tokens per segment for a set of sweeps (0: no cutting), the number of
// segments with others after them, which have a state each, and that of the
// items a grid has to cover.
uint64_t linattn_seg_len(uint64_t tokens, bool ragged, uint32_t seqs, uint32_t heads, int sweeps,
                         int width);
uint64_t linattn_slots(uint64_t tokens, bool ragged, uint32_t seqs, uint64_t seg_len);
uint64_t linattn_items(uint64_t tokens, bool ragged, uint32_t seqs, uint64_t seg_len);
// Floats of a segment's state.
size_t linattn_state_floats(int width);

hipError_t launch_sweeps(const SweepSet &set, hipStream_t stream);
// What launch_sweeps takes for bf16 and f16 rows, and the scan of segment
// states (padded to `width` x `width`) that every kind of sweep shares.
void launch_sweeps_split(const SweepSet &set, int width, hipStream_t stream);
void launch_segment_scan(const SweepSet &set, int width, hipStream_t stream);

// Sums the `share` consecutive heads of float rows into rows of `dtype`.  Of a
// packed batch, the rows before the last end: no sweep has written the others.
struct HeadSum {
    const float *src;            // [seqs][tokens][heads * share][width], dense
    Rows dst;                    // share unused
    uint64_t tokens, seqs;
    const uint32_t *last_end;    // of a packed batch, or null
    bool clear;                  // zeros in the rows after it
    uint32_t heads, share;
    int width, dtype;
};
hipError_t launch_head_sum(const HeadSum &h, hipStream_t stream);

struct StepArgs {
    Rows q, k, v, out;           // seq is the stride of a row
    int dtype, dk, dv;
    uint32_t rows, heads;
    const float *log_decay;
    float scale;
    const float *state;
    float *state_out;
    uint64_t pool;
    const int32_t *slots;
};
hipError_t launch_linattn_step(const StepArgs &a, hipStream_t stream);

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------

typedef float f32x4 __attribute__((ext_vector_type(4)));

// e^(g n) for n >= 0, with e^(g 0) = 1 for every g (a head without memory
// has g = -inf), as the nearest float and what that leaves.  A state is
// decayed once a chunk by the same power: with the rounded one alone its
// error would grow with every chunk (2^-25 of the state each time, and always
// to one side), so states are multiplied by both parts.
struct Power {
    float hi, lo;
};

__device__ __forceinline__ Power decay_power(float g, double n)
{
    const double x = n == 0.0 ? 1.0 : exp((double)g * n);
    const float hi = (float)x;
    const float lo = (float)(x - (double)hi);
    return Power{hi, lo == lo ? lo : 0.f};      // hi may be infinite
}

__device__ __forceinline__ float decayed(float x, Power p)
{
    // An infinity times lo, which may be zero or of the other sign, is left out.
    const float most = 3.402823466e38f;
    return __builtin_fmaf(x, p.hi, __builtin_amdgcn_fmed3f(x, -most, most) * p.lo);
}

template <class T>
__device__ __forceinline__ const T *row_ptr(const Rows &r, uint64_t seq, uint64_t tok, uint32_t head)
{
    return static_cast<const T *>(r.p) + (int64_t)seq * r.seq + (int64_t)tok * r.tok +
           (int64_t)(head / r.share) * r.head;
}

// Which sequence, and which segment of it, a workgroup has.
struct Place {
    uint32_t seq;
    uint64_t first;      // token of the packed batch the sequence starts at (0 when dense)
    uint64_t len;        // tokens of the sequence
    uint64_t lo, hi;     // the segment, in the sweep's order
    uint32_t slot0;      // where the state of the sequence's first segment is
    bool last;
};

// Sequence i of a packed batch.  Ends past the batch are cut to it and a
// sequence that ends before it starts has no tokens, so that no list of ends
// reaches outside the rows.  With falling ends two sequences may hold the same
// rows, and a slot may be left as it was.
__device__ __forceinline__ void run_of(const uint32_t *ends, uint64_t tokens, uint32_t i,
                                       uint64_t *first, uint64_t *len)
{
    const uint64_t lo = i ? ends[i - 1] : 0u, hi = ends[i];
    const uint64_t a = lo < tokens ? lo : tokens, b = hi < tokens ? hi : tokens;
    *first = a;
    *len = b > a ? b - a : 0;
}

// The first of the ascending `ends` above x, or `n`.  One wave, 64 at a time.
__device__ __forceinline__ uint32_t first_above(const uint32_t *ends, uint32_t n, uint64_t x)
{
    uint32_t at = 0;
    while (n) {
        // Lane l looks at the last of the l-th `step`.
        const uint32_t step = (n + 63) / 64, whole = n / step, l = threadIdx.x & 63;
        const uint64_t hit = __ballot(l < whole && ends[at + (l < whole ? l : 0) * step + step - 1] > x);
        const uint32_t skip = hit ? (uint32_t)__ffsll((unsigned long long)hit) - 1 : whole;
        at += skip * step;
        n = hit ? step - 1 : n - whole * step;
    }
    return at;
}

// A sequence of n > 1 segments has n - 1 slots, from slot0 on, for the states
// of all but the last.  In a packed batch, a segment of L tokens holds one
// multiple of L among the batch's tokens, and that over L is its slot: so a
// slot's sequence is found by its token, and slots and items do not depend on
// where sequences end.  Items are each sequence's last segment, then the
// slots'; those of a dense batch are all segments in order.  `cut`: only what
// has a slot, where states are summed.  False: the item has no segment.
__device__ __forceinline__ bool place_of(const SweepSet &set, uint32_t item, bool cut, Place *p)
{
    const uint64_t L = set.seg_len;
    uint64_t s = 0, segs = 1;
    if (!set.ends) {
        p->first = 0;
        p->len = set.tokens;
        segs = L && p->len ? (p->len + L - 1) / L : 1;
        const uint64_t n = cut ? segs - 1 : segs;
        p->seq = (uint32_t)(item / n);
        s = item % n;
        p->slot0 = p->seq * (uint32_t)(segs - 1);
        if (p->seq >= set.seqs)
            return false;
    } else if (cut || item >= set.seqs) {
        const uint32_t slot = cut ? item : item - set.seqs;
        const uint64_t x = slot * L;
        if (slot >= set.slots)
            return false;
        p->seq = first_above(set.ends, set.seqs, x);
        if (p->seq >= set.seqs)
            return false;
        run_of(set.ends, set.tokens, p->seq, &p->first, &p->len);
        p->slot0 = (uint32_t)((p->first + L - 1) / L);
        s = slot - p->slot0;
        if (x < p->first || (s + 1) * L >= p->len)
            return false;
    } else {
        p->seq = item;
        run_of(set.ends, set.tokens, p->seq, &p->first, &p->len);
        p->slot0 = L ? (uint32_t)((p->first + L - 1) / L) : 0;
        segs = L && p->len ? (p->len + L - 1) / L : 1;
        s = segs - 1;
    }
    p->lo = s * L;
    p->hi = L && p->lo + L < p->len ? p->lo + L : p->len;
    p->last = p->hi == p->len;
    return true;
}

}  // namespace libscan
