// linattn_kernels.hip -- linear attention with a decay for each head: the scan
// of segment states, the sum of shared heads' gradients, and single tokens.
// linattn.hpp has the mathematics, linattn_split.hip the sweeps.
#include "linattn.hpp"

#include "../../include/libscan.h"

namespace libscan {

namespace {

template <class T>
__device__ __forceinline__ float to_f32(T x) { return (float)x; }

// The scan of a sequence's segment states, (l, S) o (r, U) = (l r, r S + U),
// each thread four elements of the state: a segment's slot is left with what
// the next one reads.  The workgroups of a sequence's first slot do it.
template <int D>
__global__ __launch_bounds__(256) void segment_scan_kernel(const SweepSet set)
{
    const uint32_t head = blockIdx.y;
    constexpr uint32_t PARTS = D * D / 1024;
    const uint32_t sweep = blockIdx.z;
    const uint64_t L = set.seg_len;
    Place pl;
    if (!place_of(set, blockIdx.x / PARTS, true, &pl) || pl.lo != 0 || pl.len <= kFewSegments * L)
        return;
    const uint64_t slots = (pl.len + L - 1) / L - 1;
    const Power w = decay_power(set.log_decay[head], (double)L);
    f32x4 *p = reinterpret_cast<f32x4 *>(
                   set.seg + (((uint64_t)sweep * set.slots + pl.slot0) * set.heads + head) * (D * D)) +
               blockIdx.x % PARTS * 256 + threadIdx.x;
    const uint64_t step = (uint64_t)set.heads * (D * D) / 4;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    constexpr int AHEAD = 8;            // loads in flight ahead of the chain
    for (uint64_t s = 0; s < slots; s += AHEAD) {
        f32x4 own[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            own[i] = s + i < slots ? p[(s + i) * step] : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (s + i < slots) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[e] = decayed(sum[e], w) + own[i][e];
                p[(s + i) * step] = sum;
            }
    }
}

// dst = the sum over each `share` consecutive heads of src, in order.
template <class T>
__global__ __launch_bounds__(256) void head_sum_kernel(const HeadSum h)
{
    const uint64_t per = (uint64_t)h.heads * h.width;
    const uint64_t all = h.seqs * h.tokens * per;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (uint64_t)gridDim.x * 256) {
        const uint64_t row = i / per, head = i % per / h.width;
        const bool outside = h.last_end && row >= *h.last_end;
        if (outside && !h.clear)
            return;
        const int c = (int)(i % h.width);
        const float *src = h.src + (row * h.heads + head) * h.share * h.width + c;
        float x = 0.f;
        for (uint32_t k = 0; k < h.share && !outside; ++k)
            x += src[(uint64_t)k * h.width];
        T *dst = static_cast<T *>(const_cast<void *>(h.dst.p));
        dst[(int64_t)(row / h.tokens) * h.dst.seq + (int64_t)(row % h.tokens) * h.dst.tok +
            (int64_t)head * h.dst.head + c] = (T)x;
    }
}

// Single tokens.  A workgroup has COLS = 4 LPR (or LPR) columns of one row's
// and head's state: LPR lanes cover a row of them, 256 / LPR rows at a time,
// so every load and store is 16 bytes a lane.  Each thread adds up its rows'
// part of the output; the row groups are added in LDS in a fixed order.
//
// The state is read and written once, which bounds it: 256 rows of 32 heads
// of 128 x 128 take 196 us, 5.5 TB/s (a copy: 6.8).  PAST: the state is past
// what the caches hold from one step to the next, and is marked as such; all
// of a thread's rows are then read at once.  Both ways, in us for 128, 192,
// 256, 384 and 512 MiB: 43, 62, 89, 166, 214 kept, 51, 76, 98, 146, 196 past.
// Rows that are no multiple of 16 bytes share their lines and are always kept
// (484 MiB of 128 x 121: 371 us kept, 638 past).
// Four rows at a time are as fast as eight or 16 where it is kept (43, 43 and
// 46 us for 128 MiB), the first four asked for before q and k.  Widths of 64
// leave half of the lanes without columns and move 5.2 to 5.7 TB/s all the
// same (512 MiB of 128 x 64: 206 us), those of 32 3.7.
template <class T, int V, int LPR, bool PAST>
__global__ __launch_bounds__(256) void step_kernel(const StepArgs a)
{
    constexpr int COLS = LPR * V, GROUPS = 256 / LPR, BATCH = PAST ? kLinattnWidth / GROUPS : 4;
    __shared__ float s_q[kLinattnWidth], s_k[kLinattnWidth];
    __shared__ float s_o[GROUPS][COLS];
    const uint32_t row = blockIdx.x, head = blockIdx.y;
    const int c0 = blockIdx.z * COLS, lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int col = c0 + lane * V;
    T *out = static_cast<T *>(const_cast<void *>(a.out.p)) + (int64_t)row * a.out.seq +
             (int64_t)head * a.out.head;
    const int64_t slot = a.slots ? (int64_t)a.slots[row] : (int64_t)row;
    if (slot < 0 || (uint64_t)slot >= a.pool) {       // an idle row
        if (threadIdx.x < COLS && c0 + (int)threadIdx.x < a.dv)
            out[c0 + threadIdx.x] = (T)0.f;
        return;
    }
    const uint64_t base = ((uint64_t)slot * a.heads + head) * ((uint64_t)a.dk * a.dv) + col;
    const float *src = a.state + base;
    float *dst = a.state_out + base;
    const bool own = col < a.dv;
    // The first rows are asked for ahead of all else.
    typedef float Row __attribute__((ext_vector_type(V)));
    Row x[BATCH];
    const auto read = [&](int from) {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int r = from + j * GROUPS;
            if (!own || r >= a.dk)
                continue;
            const Row *at = reinterpret_cast<const Row *>(src + (int64_t)r * a.dv);
            x[j] = PAST ? __builtin_nontemporal_load(at) : *at;
        }
    };
    read(group);
    const T *q = row_ptr<T>(a.q, row, 0, head), *k = row_ptr<T>(a.k, row, 0, head);
    const T *v = row_ptr<T>(a.v, row, 0, head);
    if ((int)threadIdx.x < a.dk) {
        s_q[threadIdx.x] = to_f32(q[threadIdx.x]) * a.scale;
        s_k[threadIdx.x] = to_f32(k[threadIdx.x]);
    }
    const Power w = decay_power(a.log_decay[head], 1.0);
    float vv[V], o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        vv[e] = col + e < a.dv ? to_f32(v[col + e]) : 0.f;
        o[e] = 0.f;
    }
    __syncthreads();
    for (int from = group; from < a.dk; from += BATCH * GROUPS) {
        if (from != group)
            read(from);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int r = from + j * GROUPS;
            if (!own || r >= a.dk)
                continue;
            const float kr = s_k[r], qr = s_q[r];
            Row y;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                y[e] = decayed(x[j][e], w) + kr * vv[e];
                o[e] += qr * y[e];
            }
            Row *at = reinterpret_cast<Row *>(dst + (int64_t)r * a.dv);
            if (PAST)
                __builtin_nontemporal_store(y, at);
            else
                *at = y;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        s_o[group][lane * V + e] = o[e];
    __syncthreads();
    if (threadIdx.x < COLS && c0 + (int)threadIdx.x < a.dv) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
            x += s_o[i][threadIdx.x];
        out[c0 + threadIdx.x] = (T)x;
    }
}

template <class T>
void run_step(const StepArgs &a, hipStream_t stream)
{
    const bool aligned = (((uintptr_t)a.state | (uintptr_t)a.state_out) & 15) == 0;
    const unsigned v = a.dv % 4 == 0 && aligned ? 4 : 1;
    const auto blocks = [&](int cols) { return (unsigned)((a.dv + cols - 1) / cols); };
    // Narrow slabs where whole ones would leave compute units idle.
    const bool narrow = (uint64_t)a.rows * a.heads < 512;
    const bool past = (uint64_t)a.rows * a.heads * a.dk * a.dv > (256u << 20) / sizeof(float);
    if (v == 4) {
        if (narrow)
            step_kernel<T, 4, 8, false><<<dim3(a.rows, a.heads, blocks(32)), 256, 0, stream>>>(a);
        else if (past)
            step_kernel<T, 4, 32, true><<<dim3(a.rows, a.heads, blocks(128)), 256, 0, stream>>>(a);
        else
            step_kernel<T, 4, 32, false><<<dim3(a.rows, a.heads, blocks(128)), 256, 0, stream>>>(a);
    } else {
        step_kernel<T, 1, 32, false><<<dim3(a.rows, a.heads, blocks(32)), 256, 0, stream>>>(a);
    }
}

}  // namespace

size_t linattn_state_floats(int width) { return width <= 64 ? 64 * 64 : 128 * 128; }

uint64_t linattn_seg_len(uint64_t tokens, bool ragged, uint32_t seqs, uint32_t heads, int sweeps,
                         int width)
{
    // About one workgroup for every place on the GPU.  Those of 128 columns
    // have two a compute unit, f32's one (93 KB of LDS); those of 64 have
    // three, f32's two, and take as long with four.  For 256, 512, 768 and
    // 1024 workgroups, in us:
    //   bf16 of 128  4 x 4096 x 16  134 119 144 140    gradient of 8192 x 8  113 104 110 110
    //   f16  of 128                 180 153 184 169                          149 133 135 134
    //   f32  of 128  4 x 2048 x 16  161 168 168 164                  4096    133 148 147 147
    //   bf16 of 64                   92  66  67  67                           78  60  53  52
    //   f16  of 64                  126  87  84  85                          108  79  66  65
    //   f32  of 64                   95  72  71  71                           90  69  68  68
    // f32's of 128 are counted as the others: 256 would take 215 for 174 in
    // gradients of five packed documents, 12 heads, whose lengths differ.
    // Segments of under 256 tokens would move more of states than of rows.
    const uint64_t places = width <= 64 ? 1024 : 512, lines = (uint64_t)heads * sweeps;
    if (ragged) {
        uint64_t share = (tokens * lines + places - 1) / places;
        // Enough sequences as they are: only what is far longer than its
        // share is cut.  In shares, in three and never, in us: 37 prompts of
        // 600 tokens on average, 24 heads, f16: 297, 258, 252; 200 of 400,
        // 8 heads of 64: 148, 134, 131; 40 of 2000, 16 heads: 478, 456, 448;
        // one of 12000 among 140 of 200, 16 heads: 364, 569, 968.
        if (seqs * lines >= places)
            share *= 3;
        share = (share + 63) / 64 * 64;
        if (share < 256)
            share = 256;
        return tokens > share ? share : 0;
    }
    uint64_t segs = places / (lines * seqs);
    if (segs > tokens / 256)
        segs = tokens / 256;
    return segs > 1 ? ((tokens + segs - 1) / segs + 63) / 64 * 64 : 0;
}

uint64_t linattn_slots(uint64_t tokens, bool ragged, uint32_t seqs, uint64_t seg_len)
{
    if (!seg_len)
        return 0;
    // A token is left behind the last segment that has a slot.
    return ragged ? (tokens - 1 + seg_len - 1) / seg_len : seqs * ((tokens + seg_len - 1) / seg_len - 1);
}

uint64_t linattn_items(uint64_t tokens, bool ragged, uint32_t seqs, uint64_t seg_len)
{
    return seqs + linattn_slots(tokens, ragged, seqs, seg_len);
}

void launch_segment_scan(const SweepSet &set, int width, hipStream_t stream)
{
    const dim3 grid((unsigned)(width * width / 1024) * set.slots, set.heads, (unsigned)set.count);
    if (width == 64)
        segment_scan_kernel<64><<<grid, 256, 0, stream>>>(set);
    else
        segment_scan_kernel<128><<<grid, 256, 0, stream>>>(set);
}

hipError_t launch_sweeps(const SweepSet &set, hipStream_t stream)
{
    int width = 0;
    for (int i = 0; i < set.count; ++i) {
        width = set.s[i].m > width ? set.s[i].m : width;
        width = set.s[i].n > width ? set.s[i].n : width;
    }
    width = width <= 64 ? 64 : 128;
    launch_sweeps_split(set, width, stream);
    return hipGetLastError();
}

hipError_t launch_head_sum(const HeadSum &h, hipStream_t stream)
{
    const uint64_t n = h.seqs * h.tokens * h.heads * (uint64_t)h.width;
    if (n == 0)
        return hipSuccess;
    // A grid holds fewer than 2^32 threads.
    const unsigned blocks = (unsigned)(n < ((uint64_t)1 << 31) ? (n + 255) / 256 : 1u << 23);
    switch (h.dtype) {
    case LIBSCAN_F32: head_sum_kernel<float><<<blocks, 256, 0, stream>>>(h); break;
    case LIBSCAN_BF16: head_sum_kernel<__bf16><<<blocks, 256, 0, stream>>>(h); break;
    default: head_sum_kernel<_Float16><<<blocks, 256, 0, stream>>>(h); break;
    }
    return hipGetLastError();
}

hipError_t launch_linattn_step(const StepArgs &a, hipStream_t stream)
{
    switch (a.dtype) {
    case LIBSCAN_F32: run_step<float>(a, stream); break;
    case LIBSCAN_BF16: run_step<__bf16>(a, stream); break;
    default: run_step<_Float16>(a, stream); break;
    }
    return hipGetLastError();
}

}  // namespace libscan
