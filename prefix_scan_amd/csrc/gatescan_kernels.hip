// gatescan_kernels.hip -- the gated recurrence over sequences and for single
// tokens (gatescan.hpp, gatescan_tile.hpp).
#include "gatescan_tile.hpp"

namespace libscan {

namespace {

// One token of each row: out = h = a h + b.  A thread has 16 bytes of a row's
// channels; bound by the states' bytes, and by the launch when rows are few.
template <class T, int FORM, bool BLEND>
__global__ __launch_bounds__(256) void gate_step_kernel(GateStepArgs p)
{
    typedef Unpack<T> U;
    constexpr int V = kPiece<T>;
    const uint64_t pieces = (p.width + V - 1) / V, all = p.rows * pieces;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (uint64_t)gridDim.x * 256) {
        const uint64_t r = i / pieces, c = i % pieces * V;
        const int n = p.width - c < (uint64_t)V ? (int)(p.width - c) : V;
        const int64_t slot = p.slots ? p.slots[r] : (int64_t)r;
        T *const out = static_cast<T *>(p.out) + (int64_t)r * p.out_seq + c;
        if (slot < 0 || (uint64_t)slot >= p.pool) {
            store_piece<T>(out, piece_t{0, 0, 0, 0}, n);
            continue;
        }
        const piece_t g = load_piece<T>(static_cast<const T *>(p.gate.p) + (int64_t)r * p.gate.seq + c, n);
        const piece_t x = load_piece<T>(static_cast<const T *>(p.x.p) + (int64_t)r * p.x.seq + c, n);
        float h[V];
        load_floats<V>(p.state + slot * p.width + c, n, h);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const Gate w = gate_of<FORM, sizeof(T) == 4>(U::get(g, e));
            const float v = U::get(x, e);
            h[e] = __builtin_fmaf(w.a, h[e], BLEND ? w.rest * v : v);
        }
        store_floats<V>(p.state_out + slot * p.width + c, n, h);
        store_piece<T>(out, U::pack(h), n);
    }
}

template <class T>
hipError_t run_gate_step(const GateStepArgs &a, hipStream_t stream)
{
    const uint64_t all = a.rows * ((a.width + kPiece<T> - 1) / kPiece<T>);
    const unsigned grid = (unsigned)(all < (256ull << 20) ? (all + 255) / 256 : 1u << 20);
#define LIBSCAN_GATE(FORM)                                                                        \
    if (a.form == FORM) {                                                                         \
        if (a.blend)                                                                              \
            gate_step_kernel<T, FORM, true><<<grid, 256, 0, stream>>>(a);                         \
        else                                                                                      \
            gate_step_kernel<T, FORM, false><<<grid, 256, 0, stream>>>(a);                        \
    }
    LIBSCAN_GATE(GATESCAN_DECAY)
    LIBSCAN_GATE(GATESCAN_LOG)
    LIBSCAN_GATE(GATESCAN_SIGMOID)
#undef LIBSCAN_GATE
    return hipGetLastError();
}

}  // namespace

bool gate_grid(int dtype, bool grad, bool packed, uint32_t seqs, uint64_t tokens, uint64_t width,
               uint32_t *blocks, uint32_t *chains, uint32_t *tiles)
{
    const uint64_t c = (uint64_t)gate_channels(dtype), t = (uint64_t)gate_tile(dtype, grad);
    const uint64_t b = (width + c - 1) / c, most = (1u << 24) - 1;      // 2^32 threads are no grid
    const uint64_t k = tokens ? (tokens + t - 1) / t : 1, lines = packed ? 1 : seqs;
    if (b > most || k > most || b * lines > most || b * lines * k > most)
        return false;
    *blocks = (uint32_t)b;
    *chains = (uint32_t)(b * lines);
    *tiles = (uint32_t)k;
    return true;
}

bool gate_far(uint32_t chains) { return chains < 128; }

size_t gate_desc_bytes(int dtype, uint32_t chains, uint32_t tiles)
{
    return tiles > 1 ? kGateCounterBytes + (size_t)chains * tiles * 2 * gate_channels(dtype) * sizeof(uint64_t) : 0;
}

hipError_t launch_gatescan(const GateArgs &a, hipStream_t stream)
{
    switch (a.dtype) {
    case LIBSCAN_F32: return launch_gate_tiles<float, false>(a, stream);
    case LIBSCAN_BF16: return launch_gate_tiles<__bf16, false>(a, stream);
    default: return launch_gate_tiles<_Float16, false>(a, stream);
    }
}

hipError_t launch_gatescan_step(const GateStepArgs &a, hipStream_t stream)
{
    switch (a.dtype) {
    case LIBSCAN_F32: return run_gate_step<float>(a, stream);
    case LIBSCAN_BF16: return run_gate_step<__bf16>(a, stream);
    default: return run_gate_step<_Float16>(a, stream);
    }
}

}  // namespace libscan
