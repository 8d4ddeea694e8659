// libscan_api.hip -- the C ABI of include/libscan.h: argument checks,
// scratch carving, kernel selection, and the optional host read-back of a
// total or count.  All GPU work is enqueued on the caller's stream.
#include "../../include/libscan.h"
#include "embed.hpp"
#include "gatescan.hpp"
#include "launch.hpp"
#include "linattn.hpp"
#include "penalty.hpp"
#include "sample.hpp"
#include "scratch_state.hpp"

#include <stdio.h>
#include <string.h>

#include <mutex>

using namespace libscan;

namespace {

thread_local hipError_t g_last_hip = hipSuccess;

int hip_status(hipError_t e)
{
    if (e == hipSuccess)
        return LIBSCAN_OK;
    g_last_hip = e;
    return LIBSCAN_ERR_HIP;
}

bool misaligned4(const void *p) { return ((uintptr_t)p & 3u) != 0; }

// Carve the aligned scratch view; false if the buffer cannot hold `body`
// bytes after the header.
bool carve(void *scratch, size_t scratch_bytes, size_t body, Scratch *out)
{
    const uintptr_t p = (uintptr_t)scratch;
    const uintptr_t a = (p + kScratchAlign - 1) & ~(uintptr_t)(kScratchAlign - 1);
    const size_t slack = (size_t)(a - p);
    if (scratch_bytes < slack)
        return false;
    const size_t usable = scratch_bytes - slack;
    if (usable < kHeaderBytes + body)
        return false;
    out->base = reinterpret_cast<uint8_t *>(a);
    out->bytes = usable;
    out->ticket_ptr = reinterpret_cast<uint64_t *>(out->base);
    out->desc_ptr = reinterpret_cast<uint64_t *>(out->base + kHeaderBytes);
    return true;
}

// ---------------------------------------------------------------------------
// Scratch state tracking (scratch_state.hpp): before each call, clear with a
// fill kernel on the call's stream whatever state the call will read that it
// cannot vouch for.
// ---------------------------------------------------------------------------
StateTable g_states;

// Whether `stream` is recording a HIP graph right now.
bool stream_capturing(hipStream_t stream)
{
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(stream, &st) != hipSuccess)
        return false;
    return st == hipStreamCaptureStatusActive;
}

hipError_t apply_plan(const Scratch &s, const ClearPlan &p, size_t state, hipStream_t stream)
{
    if (p.header)
        return launch_fill_zero(s.base, kHeaderBytes + state, stream);
    if (p.bytes)
        return launch_fill_zero(s.body() + p.from, p.bytes, stream);
    return hipSuccess;
}

// launch: the call's last launch's number among the buffer's since its state was cleared.
hipError_t prepare_state(const Scratch &s, int kind, uint64_t sig, size_t state,
                         uint64_t launches, hipStream_t stream, uint64_t *launch = nullptr)
{
    const uintptr_t key = (uintptr_t)s.base;
    const ClearPlan p = g_states.prepare(key, kind, sig, state, launches, stream_capturing(stream), launch);
    const hipError_t e = apply_plan(s, p, state, stream);
    if (e != hipSuccess)
        g_states.forget(key);
    return e;
}

size_t with_header(size_t body) { return (kScratchAlign - 1) + kHeaderBytes + body; }

// The three-pass depth: d = min(b, floor(log2 n), kMaxForkDepth), or the
// automatic choice for b = -1.  Every depth gives the same bits, so the cap
// (which bounds the grid and the sums array) never changes a result.
constexpr unsigned kMaxForkDepth = 24;

unsigned threepass_depth(uint64_t n, int fork_depth)
{
    const unsigned lg = floor_log2(n ? n : 1);
    unsigned d = fork_depth < 0 ? threepass_auto_depth(n) : (unsigned)fork_depth;
    if (d > lg)
        d = lg;
    if (d > kMaxForkDepth)
        d = kMaxForkDepth;
    return d;
}

// Copies the u32 result at `dev` to `host` and waits for the stream.
int read_back(uint32_t *host, const uint32_t *dev, hipStream_t stream)
{
    hipError_t e = hipMemcpyAsync(host, dev, sizeof(uint32_t), hipMemcpyDeviceToHost, stream);
    if (e != hipSuccess)
        return hip_status(e);
    return hip_status(hipStreamSynchronize(stream));
}

int read_back64(uint64_t *host, const uint64_t *dev, hipStream_t stream)
{
    hipError_t e = hipMemcpyAsync(host, dev, sizeof(uint64_t), hipMemcpyDeviceToHost, stream);
    if (e != hipSuccess)
        return hip_status(e);
    return hip_status(hipStreamSynchronize(stream));
}

int report_value64(uint64_t *host, uint64_t *dev, uint64_t value, hipStream_t stream)
{
    if (dev) {
        hipError_t e = launch_fill_u64(dev, value, stream);
        if (e != hipSuccess)
            return hip_status(e);
    }
    if (host) {
        hipError_t e = hipStreamSynchronize(stream);
        if (e != hipSuccess)
            return hip_status(e);
        *host = value;
    }
    return LIBSCAN_OK;
}

bool misaligned8(const void *p) { return ((uintptr_t)p & 7u) != 0; }

// A fixed result (the operator's identity) to report for an empty input.
int report_value(uint32_t *host, uint32_t *dev, uint32_t value, hipStream_t stream)
{
    if (dev) {
        hipError_t e = launch_fill_u32(dev, value, stream);
        if (e != hipSuccess)
            return hip_status(e);
    }
    if (host) {
        hipError_t e = hipStreamSynchronize(stream);
        if (e != hipSuccess)
            return hip_status(e);
        *host = value;
    }
    return LIBSCAN_OK;
}

int report_zero(uint32_t *host, uint32_t *dev, hipStream_t stream)
{
    return report_value(host, dev, 0u, stream);
}

// Identities of the LIBSCAN_OP_* operators.
uint32_t op_identity(int op)
{
    static const uint32_t id[9] = {0u, 1u, 0xFFFFFFFFu, 0u, 0u, 0xFFFFFFFFu, 0u, 0x7FFFFFFFu,
                                   0x80000000u};
    return id[op];
}

uint64_t op_identity64(int op)
{
    static const uint64_t id[9] = {0u, 1u, ~0ull, 0u, 0u, ~0ull, 0u, 0x7FFFFFFFFFFFFFFFull,
                                   0x8000000000000000ull};
    return id[op];
}

constexpr uint64_t kAutoTileMaxN = 1ull << 24;

int scan_common(uint32_t *data, uint64_t n, int inclusive, int algo, int fork_depth,
                uint32_t *total_host, uint32_t *total_dev, void *scratch, size_t scratch_bytes,
                hipStream_t stream)
{
    if (algo < LIBSCAN_ALGO_AUTO || algo > LIBSCAN_ALGO_LOOKBACK_TILE)
        return LIBSCAN_ERR_ARG;
    if (fork_depth < -1 || fork_depth > 40)
        return LIBSCAN_ERR_ARG;
    if (algo != LIBSCAN_ALGO_THREEPASS && fork_depth != -1)
        return LIBSCAN_ERR_ARG;
    if (n > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(data) || misaligned4(total_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_zero(total_host, total_dev, stream);
    if (!data || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes,
               scan_ex_scratch_bytes(n, algo, fork_depth) - with_header(0), &s))
        return LIBSCAN_ERR_SCRATCH;
    uint32_t *tot = total_dev ? total_dev : s.total_slot();
    // Automatic choice, from measurements on MI355X: up to 2^24 elements the
    // grid that runs one tile per workgroup (512 x 32) finishes first -- too
    // few tiles per workgroup for two in flight to pay (2^24: 27.7 against
    // 31.3 us); from 2^25 on, the pipelined kernel (2^28: 342 against 407 us).
    if (algo == LIBSCAN_ALGO_AUTO)
        algo = n <= kAutoTileMaxN ? LIBSCAN_ALGO_LOOKBACK_TILE : LIBSCAN_ALGO_LOOKBACK;
    hipError_t e;
    if (algo == LIBSCAN_ALGO_THREEPASS) {
        const unsigned d = threepass_depth(n, fork_depth);
        e = prepare_state(s, kKindData, 0, 0, 0, stream);
        if (e == hipSuccess)
            e = launch_scan_threepass(data, n, inclusive != 0, d, s, tot, stream);
    } else {
        e = prepare_state(s, kKindDesc, 0, scan_lookback_body_bytes(n, 3), 1, stream);
        if (e != hipSuccess)
            return hip_status(e);
        e = launch_scan_lookback(data, n, inclusive != 0, algo != LIBSCAN_ALGO_LOOKBACK_TILE, s,
                                 tot, stream);
    }
    if (e != hipSuccess)
        return hip_status(e);
    if (total_host)
        return read_back(total_host, tot, stream);
    return LIBSCAN_OK;
}

// ---------------------------------------------------------------------------
// scan_u32_noalloc: the scan with its scratch in a static device array, for
// callers that cannot allocate.  Each device holds its own copy of the
// array, at its own address; host code reaches it only through the address
// hipGetSymbolAddress returns for the device (the array's name is a host-side
// stand-in, not a device address).  The array keeps the chained carry's
// header and the descriptors of the default tile shapes: up to
// kNoallocTiles tiles of at least kDefaultScanTile elements, so n up to
// LIBSCAN_NOALLOC_MAX_N whatever the array's 16-byte phase.
// ---------------------------------------------------------------------------
constexpr uint64_t kNoallocTiles = (LIBSCAN_NOALLOC_MAX_N + 3 + kDefaultScanTile - 1) / kDefaultScanTile;
constexpr size_t kNoallocBody = (kNoallocTiles * sizeof(uint64_t) + kScratchAlign - 1) /
                                kScratchAlign * kScratchAlign;
constexpr size_t kNoallocBytes = kHeaderBytes + kNoallocBody;
static_assert(kNoallocBytes == LIBSCAN_NOALLOC_SCRATCH_BYTES, "the header states the array's size");

constexpr int kNoallocMaxDevices = 64;

// Per device: the array's address and what the last call left in it.  A
// fixed table (no heap), guarded by a mutex.
struct NoallocDevice {
    void *ptr;             // device address of the array, or null before set-up
    StateRecord rec;
    bool captured;         // used under graph capture: never trust its state again
};
std::mutex g_noalloc_mu;
NoallocDevice g_noalloc[kNoallocMaxDevices];


// ---------------------------------------------------------------------------
// Linear attention: checks and the sweeps of a call (linattn.hpp).
// ---------------------------------------------------------------------------

size_t element_bytes(int dtype) { return dtype == LIBSCAN_F32 ? 4 : 2; }

bool bad_type(int dtype) { return dtype < LIBSCAN_F32 || dtype > LIBSCAN_F16; }

// The shape without the flag, which only sequences have, as *clear.
int take_shape(const linattn_shape_t *s, linattn_shape_t *to, bool *clear)
{
    if (!s)
        return LIBSCAN_ERR_NULL;
    *to = *s;
    *clear = s->dtype >= 0 && (s->dtype & LINATTN_CLEAR_REST) != 0;
    if (*clear)
        to->dtype &= ~LINATTN_CLEAR_REST;
    return LIBSCAN_OK;
}

int check_shape(const linattn_shape_t *s)
{
    if (!s)
        return LIBSCAN_ERR_NULL;
    if (bad_type(s->dtype) || s->heads == 0 || s->key_width == 0 || s->value_width == 0 ||
        s->key_width > LINATTN_MAX_WIDTH || s->value_width > LINATTN_MAX_WIDTH)
        return LIBSCAN_ERR_ARG;
    if (s->heads > 65535 || s->seqs > (1u << 24) || s->tokens > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(s->ends) || misaligned4(s->log_decay))
        return LIBSCAN_ERR_ALIGN;
    return LIBSCAN_OK;
}

// `any`: the rows hold something (else the tensor's pointer is not looked at).
int check_rows(const linattn_shape_t &s, const linattn_rows_t *r, bool any, bool output)
{
    if (!r)
        return LIBSCAN_ERR_NULL;
    if (r->heads == 0 || s.heads % r->heads != 0 || (output && r->heads != s.heads))
        return LIBSCAN_ERR_ARG;
    if ((uintptr_t)r->data % element_bytes(s.dtype) != 0)
        return LIBSCAN_ERR_ALIGN;
    if (any && !r->data)
        return LIBSCAN_ERR_NULL;
    return LIBSCAN_OK;
}

Rows rows_of(const linattn_shape_t &s, const linattn_rows_t &r)
{
    return Rows{r.data, s.ends ? 0 : r.seq_stride, r.token_stride, r.head_stride, s.heads / r.heads};
}

bool rows_aligned(const linattn_shape_t &s, const Rows &r, uint32_t width)
{
    const size_t b = element_bytes(s.dtype);
    return (uintptr_t)r.p % 16 == 0 && width * b % 16 == 0 && r.seq * (int64_t)b % 16 == 0 &&
           r.tok * (int64_t)b % 16 == 0 && r.head * (int64_t)b % 16 == 0 &&
           // a chunk of 64 within 32 bits
           r.tok >= 0 && (uint64_t)r.tok * b < ((uint64_t)1 << 25);
}

int widest(const linattn_shape_t &s)
{
    return (int)(s.key_width > s.value_width ? s.key_width : s.value_width);
}

// Everything of a set but its sweeps.
SweepSet sweep_set(const linattn_shape_t &s, int count, bool clear = false)
{
    SweepSet set = {};
    set.count = count;
    set.dtype = s.dtype;
    set.log_decay = s.log_decay;
    set.ends = s.ends;
    set.clear_from = clear && s.ends ? s.ends + s.seqs - 1 : nullptr;
    set.seqs = s.seqs;
    set.heads = s.heads;
    set.tokens = s.tokens;
    set.seg_len = linattn_seg_len(s.tokens, s.ends != nullptr, s.seqs, s.heads, count, widest(s));
    set.slots = (uint32_t)linattn_slots(s.tokens, s.ends != nullptr, s.seqs, set.seg_len);
    set.items = (uint32_t)linattn_items(s.tokens, s.ends != nullptr, s.seqs, set.seg_len);
    return set;
}

size_t segment_bytes(const linattn_shape_t &s, int count)
{
    return round_up((size_t)count * sweep_set(s, count).slots * s.heads * linattn_state_floats(widest(s)) *
                        sizeof(float),
                    kScratchAlign);
}

// Threads of a grid's side: 2^32 are refused by the launch, and by the checks
// before anything is launched.
bool past_a_grid(uint64_t groups, unsigned threads) { return groups * threads > 0xFFFFFFFFull; }

bool too_many_items(const linattn_shape_t &s, int count)
{
    return past_a_grid(sweep_set(s, count).items, widest(s) <= 64 ? 256 : 512);
}

uint64_t all_rows(const linattn_shape_t &s) { return s.ends ? s.tokens : s.tokens * s.seqs; }

// Float rows of every head, for the gradients of a tensor with shared heads.
size_t partial_bytes(const linattn_shape_t &s, uint32_t heads, uint32_t width)
{
    if (heads == s.heads)
        return 0;
    return round_up((size_t)all_rows(s) * s.heads * width * sizeof(float), kScratchAlign);
}

void out_of(const linattn_shape_t &s, Sweep &w, const linattn_rows_t &r, float *partial, uint32_t width)
{
    w.out_f32 = r.heads != s.heads;
    w.out = w.out_f32 ? partial : r.data;
    w.out_head = w.out_f32 ? (int64_t)width : r.head_stride;
    w.out_tok = w.out_f32 ? (int64_t)s.heads * width : r.token_stride;
    w.out_seq = s.ends ? 0 : (w.out_f32 ? (int64_t)s.tokens * s.heads * width : r.seq_stride);
    w.out_whole = w.out_f32 ? width % 4 == 0 && w.out_tok < (1 << 23) : rows_aligned(s, rows_of(s, r), width);
}

int check_embed(const embed_shape_t *s, const void *table, const void *ids, const void *rows, bool by_row)
{
    if (!s)
        return LIBSCAN_ERR_NULL;
    if (bad_type(s->dtype) || bad_type(s->out_dtype) || (s->id_bytes != 4 && s->id_bytes != 8) || s->width == 0)
        return LIBSCAN_ERR_ARG;
    if (s->rows > EMBED_MAX_ROWS || s->tokens > LIBSCAN_MAX_N || s->width > LIBSCAN_MAX_N ||
        (by_row && s->tokens > EMBED_MAX_ROWS))
        return LIBSCAN_ERR_SIZE;
    // The table is weight or dweight, the rows out or dout.
    if ((uintptr_t)table % element_bytes(by_row ? s->out_dtype : s->dtype) != 0 ||
        (uintptr_t)rows % element_bytes(by_row ? s->dtype : s->out_dtype) != 0 ||
        (uintptr_t)ids % (unsigned)s->id_bytes != 0)
        return LIBSCAN_ERR_ALIGN;
    if ((!table && s->rows != 0) || ((!rows || !ids) && s->tokens != 0))
        return LIBSCAN_ERR_NULL;
    return LIBSCAN_OK;
}

// ---------------------------------------------------------------------------
// Gated recurrence: checks (gatescan.hpp).
// ---------------------------------------------------------------------------

int check_gate_shape(const gatescan_shape_t *s)
{
    if (!s)
        return LIBSCAN_ERR_NULL;
    if (bad_type(s->dtype) || s->form < GATESCAN_DECAY || s->form > GATESCAN_SIGMOID ||
        (s->blend & ~1) != 0 || (s->clear_rest & ~1) != 0 || s->width == 0)
        return LIBSCAN_ERR_ARG;
    if (s->seqs > (1u << 24) || s->tokens > LIBSCAN_MAX_N || s->width > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    return misaligned4(s->ends) ? LIBSCAN_ERR_ALIGN : LIBSCAN_OK;
}

// `any`: the rows hold something (else the tensor's pointer is not looked at).
int check_gate_rows(const gatescan_shape_t &s, const gatescan_rows_t *r, bool any)
{
    if (!r)
        return LIBSCAN_ERR_NULL;
    if ((uintptr_t)r->data % element_bytes(s.dtype) != 0)
        return LIBSCAN_ERR_ALIGN;
    return any && !r->data ? LIBSCAN_ERR_NULL : LIBSCAN_OK;
}

GateRows gate_rows_of(const gatescan_shape_t &s, const gatescan_rows_t &r)
{
    return GateRows{r.data, s.ends ? 0 : r.seq_stride, r.token_stride};
}

void gate_out(const gatescan_shape_t &s, const gatescan_rows_t &r, int i, GateArgs *a)
{
    a->out[i] = r.data;
    a->out_seq[i] = s.ends ? 0 : r.seq_stride;
    a->out_tok[i] = r.token_stride;
}

// The call's grid and its scratch, prepared.
int gate_prepare(const gatescan_shape_t &s, bool grad, void *scratch, size_t scratch_bytes, GateArgs *a,
                 hipStream_t stream)
{
    a->dtype = s.dtype;
    a->form = s.form;
    a->blend = s.blend != 0;
    a->clear = s.clear_rest != 0 && s.ends;
    a->seqs = s.seqs;
    a->tokens = s.tokens;
    a->width = s.width;
    a->ends = s.ends;
    if (!gate_grid(s.dtype, grad, s.ends != nullptr, s.seqs, s.tokens, s.width, &a->blocks, &a->chains,
                   &a->tiles))
        return LIBSCAN_ERR_SIZE;
    a->far = gate_far(a->chains);
    const size_t body = gate_desc_bytes(s.dtype, a->chains, a->tiles);
    Scratch scr;
    if (!carve(scratch, scratch_bytes, body, &scr))
        return LIBSCAN_ERR_SCRATCH;
    if (body == 0)            // lines of one tile use no scratch at all
        return LIBSCAN_OK;
    a->counters = scr.desc();
    a->desc = scr.desc() + kGateCounterBytes / sizeof(uint64_t);
    // The launch's tag: its number among the buffer's launches since its state
    // was cleared, with a bit set that no epoch of the header's ticket has.
    uint64_t launch = 0;
    const hipError_t e = prepare_state(scr, kKindDesc, 0, body, 1, stream, &launch);
    a->tag = ((uint32_t)launch | (uint32_t)kMaxLaunchesBetweenClears) << 2;
    return hip_status(e);
}

}  // namespace

static __device__ __align__(256) uint8_t noalloc_scratch[kNoallocBytes];

namespace {

// The device `stream` runs on.
hipError_t device_of(hipStream_t stream, int *dev)
{
    if (stream == nullptr)
        return hipGetDevice(dev);
    hipDevice_t d = 0;
    const hipError_t e = hipStreamGetDevice(stream, &d);
    *dev = (int)d;
    return e;
}

// The array's address on `dev`, looked up once per device with that device
// current (the caller holds g_noalloc_mu).
hipError_t noalloc_ptr(int dev, void **out)
{
    NoallocDevice &d = g_noalloc[dev];
    if (!d.ptr) {
        int cur = 0;
        hipError_t e = hipGetDevice(&cur);
        if (e != hipSuccess)
            return e;
        if (cur != dev && (e = hipSetDevice(dev)) != hipSuccess)
            return e;
        void *p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(noalloc_scratch));
        if (cur != dev) {
            const hipError_t e2 = hipSetDevice(cur);
            if (e == hipSuccess)
                e = e2;
        }
        if (e != hipSuccess)
            return e;
        if (p == nullptr || ((uintptr_t)p & (kScratchAlign - 1)) != 0)
            return hipErrorInvalidSymbol;
        d.ptr = p;
        d.rec = StateRecord{kKindNone, 0, 0, 0};
        d.captured = false;
    }
    *out = d.ptr;
    return hipSuccess;
}

}  // namespace

extern "C" {

const char *libscan_strerror(int status)
{
    switch (status) {
    case LIBSCAN_OK: return "ok";
    case LIBSCAN_ERR_NULL: return "a required pointer is NULL";
    case LIBSCAN_ERR_SIZE: return "n is beyond this entry point's limit";
    case LIBSCAN_ERR_ARG: return "an argument is outside its documented range";
    case LIBSCAN_ERR_SCRATCH: return "scratch buffer is smaller than the size query's answer";
    case LIBSCAN_ERR_HIP: return hipGetErrorString(g_last_hip);
    case LIBSCAN_ERR_ALIGN: return "a pointer is not aligned to its elements";
    default: return "unknown libscan status";
    }
}

const char *libscan_version(void) { return "libscan 0.1 gfx950"; }

int libscan_scratch_init(void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (!scratch)
        return scratch_bytes ? LIBSCAN_ERR_NULL : LIBSCAN_OK;
    Scratch s;
    if (!carve(scratch, scratch_bytes, 0, &s))
        return LIBSCAN_ERR_SCRATCH;
    // The header only: the record says no body byte is trusted, so each call
    // clears the state it needs on first use.
    hipError_t e = launch_fill_zero(s.base, kHeaderBytes, stream);
    if (e != hipSuccess)
        return hip_status(e);
    g_states.zeroed((uintptr_t)s.base, stream_capturing(stream));
    return LIBSCAN_OK;
}

int libscan_scratch_captured(const void *scratch, size_t scratch_bytes)
{
    Scratch s;
    return scratch && carve(const_cast<void *>(scratch), scratch_bytes, 0, &s) &&
                   g_states.captured((uintptr_t)s.base)
               ? 1
               : 0;
}

size_t scan_scratch_bytes(uint64_t n)
{
    // Any head (0..3) fits: size for the largest.
    return with_header(scan_lookback_body_bytes(n, 3));
}

size_t scan_ex_scratch_bytes(uint64_t n, int algo, int fork_depth)
{
    if (algo == LIBSCAN_ALGO_THREEPASS) {
        return with_header(scan_threepass_body_bytes(threepass_depth(n, fork_depth)));
    }
    return scan_scratch_bytes(n);
}

int scan_exclusive_u32(uint32_t *data, uint64_t n, uint32_t *total_host, uint32_t *total_dev,
                       void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    return scan_common(data, n, 0, LIBSCAN_ALGO_AUTO, -1, total_host, total_dev, scratch,
                       scratch_bytes, stream);
}

int scan_inclusive_u32(uint32_t *data, uint64_t n, uint32_t *total_host, uint32_t *total_dev,
                       void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    return scan_common(data, n, 1, LIBSCAN_ALGO_AUTO, -1, total_host, total_dev, scratch,
                       scratch_bytes, stream);
}

int scan_u32_ex(uint32_t *data, uint64_t n, int inclusive, int algo, int fork_depth,
                uint32_t *total_host, uint32_t *total_dev, void *scratch, size_t scratch_bytes,
                hipStream_t stream)
{
    if (inclusive != 0 && inclusive != 1)
        return LIBSCAN_ERR_ARG;
    return scan_common(data, n, inclusive, algo, fork_depth, total_host, total_dev, scratch,
                       scratch_bytes, stream);
}

int scan_op_u32(uint32_t *data, uint64_t n, int op, int inclusive, uint32_t *total_host,
                uint32_t *total_dev, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (op < LIBSCAN_OP_ADD || op > LIBSCAN_OP_MAX_S || (inclusive != 0 && inclusive != 1))
        return LIBSCAN_ERR_ARG;
    if (n > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(data) || misaligned4(total_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_value(total_host, total_dev, op_identity(op), stream);
    if (!data || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, scan_lookback_body_bytes(n, 3), &s))
        return LIBSCAN_ERR_SCRATCH;
    uint32_t *tot = total_dev ? total_dev : s.total_slot();
    hipError_t e = prepare_state(s, kKindDesc, 0, scan_lookback_body_bytes(n, 3), 1, stream);
    if (e == hipSuccess)
        e = launch_scan_op(data, n, op, inclusive != 0, s, tot, stream);
    if (e != hipSuccess)
        return hip_status(e);
    if (total_host)
        return read_back(total_host, tot, stream);
    return LIBSCAN_OK;
}

size_t reduce_scratch_bytes(uint64_t n)
{
    (void)n;
    const size_t a = reduce_body_bytes(), b = reduce64_body_bytes();
    return with_header(a > b ? a : b);
}

int reduce_op_u32(const uint32_t *data, uint64_t n, int op, uint32_t *total_host,
                  uint32_t *total_dev, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (op < LIBSCAN_OP_ADD || op > LIBSCAN_OP_MAX_S)
        return LIBSCAN_ERR_ARG;
    if (n > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(data) || misaligned4(total_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_value(total_host, total_dev, op_identity(op), stream);
    if (!data || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, reduce_body_bytes(), &s))
        return LIBSCAN_ERR_SCRATCH;
    uint32_t *tot = total_dev ? total_dev : s.total_slot();
    hipError_t e = prepare_state(s, kKindData, 0, 0, 0, stream);
    if (e == hipSuccess)
        e = launch_reduce_op(data, n, op, s, tot, stream);
    if (e != hipSuccess)
        return hip_status(e);
    if (total_host)
        return read_back(total_host, tot, stream);
    return LIBSCAN_OK;
}

size_t scan_op_u64_scratch_bytes(uint64_t n)
{
    return with_header(scan64_body_bytes(n, 1));
}

int scan_op_u64(uint64_t *data, uint64_t n, int op, int inclusive, uint64_t *total_host,
                uint64_t *total_dev, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (op < LIBSCAN_OP_ADD || op > LIBSCAN_OP_MAX_S || (inclusive != 0 && inclusive != 1))
        return LIBSCAN_ERR_ARG;
    if (n > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned8(data) || misaligned8(total_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_value64(total_host, total_dev, op_identity64(op), stream);
    if (!data || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, scan64_body_bytes(n, 1), &s))
        return LIBSCAN_ERR_SCRATCH;
    uint64_t *tot = total_dev ? total_dev : s.total_slot64();
    hipError_t e = prepare_state(s, kKindDesc, 0, scan64_body_bytes(n, 1), 1, stream);
    if (e == hipSuccess)
        e = launch_scan_op64(data, n, op, inclusive != 0, s, tot, stream);
    if (e != hipSuccess)
        return hip_status(e);
    if (total_host)
        return read_back64(total_host, tot, stream);
    return LIBSCAN_OK;
}

int reduce_op_u64(const uint64_t *data, uint64_t n, int op, uint64_t *total_host,
                  uint64_t *total_dev, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (op < LIBSCAN_OP_ADD || op > LIBSCAN_OP_MAX_S)
        return LIBSCAN_ERR_ARG;
    if (n > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned8(data) || misaligned8(total_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_value64(total_host, total_dev, op_identity64(op), stream);
    if (!data || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, reduce64_body_bytes(), &s))
        return LIBSCAN_ERR_SCRATCH;
    uint64_t *tot = total_dev ? total_dev : s.total_slot64();
    hipError_t e = prepare_state(s, kKindData, 0, 0, 0, stream);
    if (e == hipSuccess)
        e = launch_reduce_op64(data, n, op, s, tot, stream);
    if (e != hipSuccess)
        return hip_status(e);
    if (total_host)
        return read_back64(total_host, tot, stream);
    return LIBSCAN_OK;
}

size_t runs_scratch_bytes(uint64_t n, uint64_t total)
{
    const size_t a = runs_body_bytes(n);
    const size_t b = (size_t)(runs_owner_all_parts(n, total) + 1) * sizeof(uint32_t);
    const size_t c = (size_t)runs_index_entries(n) * sizeof(uint32_t);
    const size_t ab = a > b ? a : b;
    return with_header(ab > c ? ab : c);
}

int runs_layout_u32(const uint32_t *counts, uint32_t *ends, uint64_t n, uint32_t *entries_host,
                    uint32_t *entries_dev, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (n > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(counts) || misaligned4(ends) || misaligned4(entries_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_value(entries_host, entries_dev, 1u, stream);
    if (!counts || !ends || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, runs_body_bytes(n), &s))
        return LIBSCAN_ERR_SCRATCH;
    uint32_t *ent = entries_dev ? entries_dev : s.total_slot();
    hipError_t e = prepare_state(s, kKindDesc, 0, runs_body_bytes(n), 1, stream);
    if (e == hipSuccess)
        e = launch_runs_ends(counts, ends, n, s, ent, stream);
    if (e != hipSuccess)
        return hip_status(e);
    if (entries_host)
        return read_back(entries_host, ent, stream);
    return LIBSCAN_OK;
}

int runs_slots_i32(int32_t *slots, uint64_t entries, hipStream_t stream)
{
    if (entries > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(slots))
        return LIBSCAN_ERR_ALIGN;
    if (entries == 0)
        return LIBSCAN_OK;
    if (!slots)
        return LIBSCAN_ERR_NULL;
    return hip_status(launch_fill_value(reinterpret_cast<uint32_t *>(slots), entries, 0xFFFFFFFFu,
                                        stream));
}

int runs_owner_u32(const uint32_t *ends, uint64_t n, const uint32_t *entry, uint64_t m,
                   int32_t *owner, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (n > LIBSCAN_MAX_N_INDEX || m > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(ends) || misaligned4(entry) || misaligned4(owner))
        return LIBSCAN_ERR_ALIGN;
    if (m == 0)
        return LIBSCAN_OK;
    if (!entry || !owner || (n != 0 && !ends))
        return LIBSCAN_ERR_NULL;
    if (n == 0)       // no run holds anything
        return hip_status(launch_fill_value(reinterpret_cast<uint32_t *>(owner), m, 0xFFFFFFFFu,
                                            stream));
    if (!scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, (size_t)runs_index_entries(n) * sizeof(uint32_t), &s))
        return LIBSCAN_ERR_SCRATCH;
    hipError_t e = prepare_state(s, kKindData, 0, 0, 0, stream);
    if (e == hipSuccess)
        e = launch_runs_owner(ends, n, entry, m, owner, s, stream);
    return hip_status(e);
}

int runs_owner_all_u32(const uint32_t *ends, uint64_t n, int32_t *owner, uint64_t total,
                       void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (n > LIBSCAN_MAX_N_INDEX || total > 0xFFFFFFFFull)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(ends) || misaligned4(owner))
        return LIBSCAN_ERR_ALIGN;
    if (total == 0)
        return LIBSCAN_OK;
    if (!owner || (n != 0 && !ends))
        return LIBSCAN_ERR_NULL;
    if (n == 0)
        return hip_status(launch_fill_value(reinterpret_cast<uint32_t *>(owner), total, 0xFFFFFFFFu,
                                            stream));
    if (!scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    const size_t body = (size_t)(runs_owner_all_parts(n, total) + 1) * sizeof(uint32_t);
    if (!carve(scratch, scratch_bytes, body, &s))
        return LIBSCAN_ERR_SCRATCH;
    hipError_t e = prepare_state(s, kKindData, 0, 0, 0, stream);
    if (e == hipSuccess)
        e = launch_runs_owner_all(ends, n, owner, total, s, stream);
    return hip_status(e);
}

size_t segscan_scratch_bytes(uint64_t n, uint64_t seg_len)
{
    return with_header(segscan_body_bytes(n, seg_len));
}

int segscan_u32(const uint32_t *in, uint32_t *out, uint64_t n, uint64_t seg_len,
                uint32_t *seg_sums, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (seg_len == 0)
        return LIBSCAN_ERR_ARG;
    if (n > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(in) || misaligned4(out) || misaligned4(seg_sums))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return LIBSCAN_OK;
    if (!in || !out || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, segscan_body_bytes(n, seg_len), &s))
        return LIBSCAN_ERR_SCRATCH;
    hipError_t e = prepare_state(s, kKindDesc, 0, segscan_body_bytes(n, seg_len), 1, stream);
    if (e != hipSuccess)
        return hip_status(e);
    return hip_status(launch_segscan(in, out, n, seg_len, seg_sums, s, stream));
}

size_t segscan_flags_scratch_bytes(uint64_t n)
{
    return with_header(segflags_body_bytes(n));
}

int segscan_flags_u32(const uint32_t *in, const int32_t *flags, uint32_t *out, uint64_t n,
                      uint32_t *seg_sums, uint32_t *nsegs_host, uint32_t *nsegs_dev,
                      void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (n > 0xFFFFFFFFull)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(in) || misaligned4(flags) || misaligned4(out) || misaligned4(seg_sums) ||
        misaligned4(nsegs_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_value(nsegs_host, nsegs_dev, 0u, stream);
    if (!in || !flags || !out || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, segflags_body_bytes(n), &s))
        return LIBSCAN_ERR_SCRATCH;
    uint32_t *cnt = nsegs_dev ? nsegs_dev : s.total_slot();
    hipError_t e = prepare_state(s, kKindDesc, 0, segflags_body_bytes(n), 1, stream);
    if (e == hipSuccess)
        e = launch_segflags(in, reinterpret_cast<const uint32_t *>(flags), out, n, seg_sums, cnt,
                            s, stream);
    if (e != hipSuccess)
        return hip_status(e);
    if (nsegs_host)
        return read_back(nsegs_host, cnt, stream);
    return LIBSCAN_OK;
}

size_t compact_scratch_bytes(uint64_t n) { return with_header(compact_body_bytes(n)); }

int compact_flags_u32(const int32_t *flags, int32_t *out_idx, uint64_t n, uint32_t *count_host,
                      uint32_t *count_dev, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (n > LIBSCAN_MAX_N_INDEX)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(flags) || misaligned4(out_idx) || misaligned4(count_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_zero(count_host, count_dev, stream);
    if (!flags || !out_idx || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, compact_body_bytes(n), &s))
        return LIBSCAN_ERR_SCRATCH;
    uint32_t *cnt = count_dev ? count_dev : s.total_slot();
    hipError_t e = prepare_state(s, kKindDesc, 0, compact_body_bytes(n), 1, stream);
    if (e != hipSuccess)
        return hip_status(e);
    e = launch_compact(flags, out_idx, n, s, cnt, stream);
    if (e != hipSuccess)
        return hip_status(e);
    if (count_host)
        return read_back(count_host, cnt, stream);
    return LIBSCAN_OK;
}

size_t radix_scratch_bytes(uint64_t n, int bits_per_pass)
{
    return with_header(radix_body_bytes(n, bits_per_pass));
}

int radix_perm_u32(const uint32_t *keys, int32_t *perm, uint64_t n, int bits_per_pass,
                   void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    if (bits_per_pass != 1 && bits_per_pass != 4)
        return LIBSCAN_ERR_ARG;
    if (n > LIBSCAN_MAX_N_INDEX)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(keys) || misaligned4(perm))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return LIBSCAN_OK;
    if (!keys || !perm || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, radix_body_bytes(n, bits_per_pass), &s))
        return LIBSCAN_ERR_SCRATCH;
    hipError_t e = prepare_state(s, kKindRadix, (n << 3) | (uint64_t)bits_per_pass,
                                 radix_state_bytes(n, bits_per_pass), bits_per_pass == 1 ? 32 : 8,
                                 stream);
    if (e != hipSuccess)
        return hip_status(e);
    return hip_status(launch_radix(keys, perm, n, bits_per_pass, s, stream));
}

int scan_u32_noalloc(uint32_t *data, uint64_t n, int inclusive, uint32_t *total_dev,
                     hipStream_t stream)
{
    if (inclusive != 0 && inclusive != 1)
        return LIBSCAN_ERR_ARG;
    if (n > LIBSCAN_NOALLOC_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(data) || misaligned4(total_dev))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return report_zero(nullptr, total_dev, stream);
    if (!data)
        return LIBSCAN_ERR_NULL;
    int dev = 0;
    hipError_t e = device_of(stream, &dev);
    if (e != hipSuccess)
        return hip_status(e);
    if (dev < 0 || dev >= kNoallocMaxDevices)
        return LIBSCAN_ERR_ARG;
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    void *ptr = nullptr;
    if ((e = noalloc_ptr(dev, &ptr)) != hipSuccess)
        return hip_status(e);
    const size_t state = (size_t)tiles_for(n, head_of(data), kDefaultScanTile) * sizeof(uint64_t);
    Scratch s;
    if (!carve(ptr, kNoallocBytes, state, &s))      // cannot fail below the limit
        return LIBSCAN_ERR_SIZE;
    NoallocDevice &d = g_noalloc[dev];
    if (stream_capturing(stream))
        d.captured = true;
    StateRecord next;
    const ClearPlan p = plan_call(d.rec, d.captured, kKindDesc, 0, state, 1, &next);
    e = apply_plan(s, p, state, stream);
    if (e != hipSuccess) {
        d.rec = StateRecord{kKindNone, 0, 0, 0};
        return hip_status(e);
    }
    d.rec = next;
    uint32_t *tot = total_dev ? total_dev : s.total_slot();
    e = launch_scan_lookback_default(data, n, inclusive != 0, n > kAutoTileMaxN, s, tot, stream);
    return hip_status(e);
}

size_t copy_scratch_bytes(uint64_t n)
{
    (void)n;
    return with_header(0);
}

int copy_u32(const uint32_t *src, uint32_t *dst, uint64_t n, void *scratch, size_t scratch_bytes,
             hipStream_t stream)
{
    if (n > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    if (misaligned4(src) || misaligned4(dst))
        return LIBSCAN_ERR_ALIGN;
    if (n == 0)
        return LIBSCAN_OK;
    if (!src || !dst || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, 0, &s))
        return LIBSCAN_ERR_SCRATCH;
    // The copy draws tiles from the header's ticket exactly as the scans do.
    hipError_t e = prepare_state(s, kKindDesc, 0, 0, 1, stream);
    if (e == hipSuccess)
        e = launch_copy(src, dst, n, s, stream);
    return hip_status(e);
}

size_t linattn_scratch_bytes(const linattn_shape_t *shape)
{
    linattn_shape_t sh;
    bool clear;
    if (take_shape(shape, &sh, &clear) != LIBSCAN_OK || check_shape(&sh) != LIBSCAN_OK || sh.seqs == 0 ||
        too_many_items(sh, 1))
        return with_header(0);
    return with_header(segment_bytes(sh, 1));
}

int linattn(const linattn_shape_t *shape, const linattn_rows_t *q, const linattn_rows_t *k,
            const linattn_rows_t *v, const float *state, const linattn_rows_t *out,
            float *state_out, void *scratch, size_t scratch_bytes, hipStream_t stream)
{
    linattn_shape_t sh;
    bool clear;
    int rc = take_shape(shape, &sh, &clear);
    if (rc != LIBSCAN_OK || (rc = check_shape(&sh)) != LIBSCAN_OK)
        return rc;
    const bool any = sh.seqs != 0 && sh.tokens != 0;
    if ((rc = check_rows(sh, q, any, false)) != LIBSCAN_OK ||
        (rc = check_rows(sh, k, any, false)) != LIBSCAN_OK ||
        (rc = check_rows(sh, v, any, false)) != LIBSCAN_OK ||
        (rc = check_rows(sh, out, any, true)) != LIBSCAN_OK)
        return rc;
    if (misaligned4(state) || misaligned4(state_out))
        return LIBSCAN_ERR_ALIGN;
    if (sh.seqs == 0)
        return LIBSCAN_OK;
    if (!sh.log_decay || !scratch)
        return LIBSCAN_ERR_NULL;
    if (state && state == state_out)
        return LIBSCAN_ERR_ARG;
    if (too_many_items(sh, 1))
        return LIBSCAN_ERR_SIZE;
    Scratch s;
    if (!carve(scratch, scratch_bytes, segment_bytes(sh, 1), &s))
        return LIBSCAN_ERR_SCRATCH;
    SweepSet set = sweep_set(sh, 1, clear);
    set.seg = reinterpret_cast<float *>(s.body());
    Sweep &w = set.s[0];
    w.a = rows_of(sh, *q);
    w.b = rows_of(sh, *k);
    w.c = rows_of(sh, *v);
    out_of(sh, w, *out, nullptr, sh.value_width);
    w.m = (int)sh.key_width;
    w.n = (int)sh.value_width;
    w.pair_scale = 1.f;
    w.out_scale = sh.scale;
    // The state enters each row's sum before out_scale.
    w.state_in = state;
    w.state_out = state_out;
    w.state_m = sh.value_width;
    w.state_n = 1;
    set.aligned = rows_aligned(sh, w.a, sh.key_width) && rows_aligned(sh, w.b, sh.key_width) &&
                  rows_aligned(sh, w.c, sh.value_width);
    hipError_t e = prepare_state(s, kKindData, 0, 0, 0, stream);
    if (e == hipSuccess)
        e = launch_sweeps(set, stream);
    return hip_status(e);
}

size_t linattn_grad_scratch_bytes(const linattn_shape_t *shape, uint32_t q_heads, uint32_t k_heads,
                                  uint32_t v_heads)
{
    linattn_shape_t sh;
    bool clear;
    if (take_shape(shape, &sh, &clear) != LIBSCAN_OK || check_shape(&sh) != LIBSCAN_OK || sh.seqs == 0 ||
        too_many_items(sh, 3))
        return with_header(0);
    return with_header(segment_bytes(sh, 3) + partial_bytes(sh, q_heads, sh.key_width) +
                       partial_bytes(sh, k_heads, sh.key_width) + partial_bytes(sh, v_heads, sh.value_width));
}

int linattn_grad(const linattn_shape_t *shape, const linattn_rows_t *dout, const linattn_rows_t *q,
                 const linattn_rows_t *k, const linattn_rows_t *v, const float *state,
                 const float *dstate_out, const linattn_rows_t *dq, const linattn_rows_t *dk,
                 const linattn_rows_t *dv, float *dstate, void *scratch, size_t scratch_bytes,
                 hipStream_t stream)
{
    linattn_shape_t sh;
    bool clear;
    int rc = take_shape(shape, &sh, &clear);
    if (rc != LIBSCAN_OK || (rc = check_shape(&sh)) != LIBSCAN_OK)
        return rc;
    const bool any = sh.seqs != 0 && sh.tokens != 0;
    if ((rc = check_rows(sh, dout, any, true)) != LIBSCAN_OK)
        return rc;
    const linattn_rows_t *in[3] = {q, k, v}, *grad[3] = {dq, dk, dv};
    for (int i = 0; i < 3; ++i) {
        if ((rc = check_rows(sh, in[i], any, false)) != LIBSCAN_OK ||
            (rc = check_rows(sh, grad[i], any, false)) != LIBSCAN_OK)
            return rc;
        if (in[i]->heads != grad[i]->heads)
            return LIBSCAN_ERR_ARG;
    }
    if (misaligned4(state) || misaligned4(dstate_out) || misaligned4(dstate))
        return LIBSCAN_ERR_ALIGN;
    if (sh.seqs == 0)
        return LIBSCAN_OK;
    if (!sh.log_decay || !scratch)
        return LIBSCAN_ERR_NULL;
    if (dstate && (dstate == state || dstate == dstate_out))
        return LIBSCAN_ERR_ARG;
    if (too_many_items(sh, 3))
        return LIBSCAN_ERR_SIZE;
    const uint32_t kw = sh.key_width, vw = sh.value_width, width[3] = {kw, kw, vw};
    size_t at = segment_bytes(sh, 3), partial[3];
    for (int i = 0; i < 3; ++i) {
        partial[i] = at;
        at += partial_bytes(sh, in[i]->heads, width[i]);
    }
    Scratch s;
    if (!carve(scratch, scratch_bytes, at, &s))
        return LIBSCAN_ERR_SCRATCH;
    SweepSet set = sweep_set(sh, 3, clear);
    set.seg = reinterpret_cast<float *>(s.body());
    const Rows rq = rows_of(sh, *q), rk = rows_of(sh, *k), rv = rows_of(sh, *v),
               ro = rows_of(sh, *dout);
    const Rows abc[3][3] = {{ro, rv, rk}, {rv, ro, rq}, {rk, rq, ro}};
    for (int i = 0; i < 3; ++i) {
        Sweep &w = set.s[i];
        w.a = abc[i][0];
        w.b = abc[i][1];
        w.c = abc[i][2];
        out_of(sh, w, *grad[i], reinterpret_cast<float *>(s.body() + partial[i]), width[i]);
        w.m = (int)(i == 2 ? kw : vw);
        w.n = (int)(i == 2 ? vw : kw);
        w.rev = w.shift = i != 0;
        // dq is scaled as a whole; the gradient of the final state reaches
        // dk and dv unscaled, so there the pairs are.
        w.pair_scale = i == 0 ? 1.f : sh.scale;
        w.out_scale = i == 0 ? sh.scale : 1.f;
        w.state_in = i == 0 ? state : dstate_out;
        w.state_out = i == 2 ? dstate : nullptr;
        w.state_m = i == 2 ? (int64_t)vw : 1;
        w.state_n = i == 2 ? 1 : (int64_t)vw;
    }
    set.aligned = rows_aligned(sh, rq, kw) && rows_aligned(sh, rk, kw) && rows_aligned(sh, rv, vw) &&
                  rows_aligned(sh, ro, vw);
    hipError_t e = prepare_state(s, kKindData, 0, 0, 0, stream);
    if (e == hipSuccess)
        e = launch_sweeps(set, stream);
    for (int i = 0; i < 3 && e == hipSuccess; ++i) {
        if (!set.s[i].out_f32)
            continue;
        HeadSum h = {};
        h.src = static_cast<const float *>(set.s[i].out);
        h.dst = rows_of(sh, *grad[i]);
        h.seqs = sh.ends ? 1 : sh.seqs;
        h.tokens = sh.tokens;
        h.last_end = sh.ends ? sh.ends + sh.seqs - 1 : nullptr;
        h.clear = clear;
        h.heads = grad[i]->heads;
        h.share = sh.heads / grad[i]->heads;
        h.width = (int)width[i];
        h.dtype = sh.dtype;
        e = launch_head_sum(h, stream);
    }
    return hip_status(e);
}

int linattn_step(const linattn_shape_t *shape, const linattn_rows_t *q, const linattn_rows_t *k,
                 const linattn_rows_t *v, const float *state, uint64_t pool, const int32_t *slots,
                 const linattn_rows_t *out, float *state_out, hipStream_t stream)
{
    int rc = check_shape(shape);
    if (rc != LIBSCAN_OK)
        return rc;
    const linattn_shape_t &sh = *shape;
    const bool any = sh.seqs != 0;
    if ((rc = check_rows(sh, q, any, false)) != LIBSCAN_OK ||
        (rc = check_rows(sh, k, any, false)) != LIBSCAN_OK ||
        (rc = check_rows(sh, v, any, false)) != LIBSCAN_OK ||
        (rc = check_rows(sh, out, any, true)) != LIBSCAN_OK)
        return rc;
    if (misaligned4(state) || misaligned4(state_out) || misaligned4(slots))
        return LIBSCAN_ERR_ALIGN;
    if (!any)
        return LIBSCAN_OK;
    if (past_a_grid(sh.seqs, 256))
        return LIBSCAN_ERR_SIZE;
    if (!sh.log_decay || ((!state || !state_out) && pool != 0))
        return LIBSCAN_ERR_NULL;
    if (pool > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    StepArgs a = {};
    // Rows are the sequences here, packed or not.
    const linattn_rows_t *rows[4] = {q, k, v, out};
    Rows *to[4] = {&a.q, &a.k, &a.v, &a.out};
    for (int i = 0; i < 4; ++i)
        *to[i] = Rows{rows[i]->data, rows[i]->seq_stride, 0, rows[i]->head_stride,
                      sh.heads / rows[i]->heads};
    a.dtype = sh.dtype;
    a.dk = (int)sh.key_width;
    a.dv = (int)sh.value_width;
    a.rows = sh.seqs;
    a.heads = sh.heads;
    a.log_decay = sh.log_decay;
    a.scale = sh.scale;
    a.state = state;
    a.state_out = state_out;
    a.pool = pool;
    a.slots = slots;
    return hip_status(launch_linattn_step(a, stream));
}

size_t gatescan_scratch_bytes(const gatescan_shape_t *shape, int grad)
{
    uint32_t blocks, chains, tiles;
    if (check_gate_shape(shape) != LIBSCAN_OK || shape->seqs == 0 ||
        !gate_grid(shape->dtype, grad != 0, shape->ends != nullptr, shape->seqs, shape->tokens, shape->width,
                   &blocks, &chains, &tiles))
        return with_header(0);
    return with_header(gate_desc_bytes(shape->dtype, chains, tiles));
}

int gatescan(const gatescan_shape_t *shape, const gatescan_rows_t *gate, const gatescan_rows_t *x,
             const float *state, const gatescan_rows_t *out, float *state_out, void *scratch,
             size_t scratch_bytes, hipStream_t stream)
{
    int rc = check_gate_shape(shape);
    if (rc != LIBSCAN_OK)
        return rc;
    const gatescan_shape_t &s = *shape;
    const bool any = s.seqs != 0 && s.tokens != 0;
    if ((rc = check_gate_rows(s, gate, any)) != LIBSCAN_OK || (rc = check_gate_rows(s, x, any)) != LIBSCAN_OK ||
        (rc = check_gate_rows(s, out, any)) != LIBSCAN_OK)
        return rc;
    if (misaligned4(state) || misaligned4(state_out))
        return LIBSCAN_ERR_ALIGN;
    if (s.seqs == 0)
        return LIBSCAN_OK;
    if (!scratch)
        return LIBSCAN_ERR_NULL;
    if (state && state == state_out)
        return LIBSCAN_ERR_ARG;
    GateArgs a = {};
    a.gate = gate_rows_of(s, *gate);
    a.x = gate_rows_of(s, *x);
    gate_out(s, *out, 0, &a);
    a.first = state;
    a.state_out = state_out;
    if ((rc = gate_prepare(s, false, scratch, scratch_bytes, &a, stream)) != LIBSCAN_OK)
        return rc;
    return hip_status(launch_gatescan(a, stream));
}

int gatescan_grad(const gatescan_shape_t *shape, const gatescan_rows_t *dout,
                  const gatescan_rows_t *gate, const gatescan_rows_t *x, const gatescan_rows_t *out,
                  const float *state, const float *dstate_out, const gatescan_rows_t *dgate,
                  const gatescan_rows_t *dx, float *dstate, void *scratch, size_t scratch_bytes,
                  hipStream_t stream)
{
    int rc = check_gate_shape(shape);
    if (rc != LIBSCAN_OK)
        return rc;
    const gatescan_shape_t &s = *shape;
    const bool any = s.seqs != 0 && s.tokens != 0;
    const gatescan_rows_t *rows[5] = {dout, gate, out, dgate, dx};
    for (const gatescan_rows_t *r : rows)
        if ((rc = check_gate_rows(s, r, any)) != LIBSCAN_OK)
            return rc;
    if ((x || s.blend) && (rc = check_gate_rows(s, x, any && s.blend)) != LIBSCAN_OK)
        return rc;
    if (misaligned4(state) || misaligned4(dstate_out) || misaligned4(dstate))
        return LIBSCAN_ERR_ALIGN;
    if (s.seqs == 0)
        return LIBSCAN_OK;
    if (!scratch)
        return LIBSCAN_ERR_NULL;
    if (dstate && (dstate == state || dstate == dstate_out))
        return LIBSCAN_ERR_ARG;
    GateArgs a = {};
    a.gate = gate_rows_of(s, *gate);
    if (s.blend)
        a.x = gate_rows_of(s, *x);
    a.dout = gate_rows_of(s, *dout);
    a.h = gate_rows_of(s, *out);
    gate_out(s, *dgate, 0, &a);
    gate_out(s, *dx, 1, &a);
    a.first = state;
    a.last = dstate_out;
    a.state_out = dstate;
    if ((rc = gate_prepare(s, true, scratch, scratch_bytes, &a, stream)) != LIBSCAN_OK)
        return rc;
    return hip_status(launch_gatescan_grad(a, stream));
}

int gatescan_step(const gatescan_shape_t *shape, const gatescan_rows_t *gate,
                  const gatescan_rows_t *x, const float *state, uint64_t pool, const int32_t *slots,
                  const gatescan_rows_t *out, float *state_out, hipStream_t stream)
{
    int rc = check_gate_shape(shape);
    if (rc != LIBSCAN_OK)
        return rc;
    const gatescan_shape_t &s = *shape;
    const bool any = s.seqs != 0;
    if ((rc = check_gate_rows(s, gate, any)) != LIBSCAN_OK || (rc = check_gate_rows(s, x, any)) != LIBSCAN_OK ||
        (rc = check_gate_rows(s, out, any)) != LIBSCAN_OK)
        return rc;
    if (misaligned4(state) || misaligned4(state_out) || misaligned4(slots))
        return LIBSCAN_ERR_ALIGN;
    if (!any)
        return LIBSCAN_OK;
    if ((!state || !state_out) && pool != 0)
        return LIBSCAN_ERR_NULL;
    if (pool > LIBSCAN_MAX_N)
        return LIBSCAN_ERR_SIZE;
    GateStepArgs a = {};
    a.gate = GateRows{gate->data, gate->seq_stride, 0};
    a.x = GateRows{x->data, x->seq_stride, 0};
    a.out = out->data;
    a.out_seq = out->seq_stride;
    a.dtype = s.dtype;
    a.form = s.form;
    a.blend = s.blend != 0;
    a.rows = s.seqs;
    a.width = s.width;
    a.state = state;
    a.state_out = state_out;
    a.pool = pool;
    a.slots = slots;
    return hip_status(launch_gatescan_step(a, stream));
}

int embed_rows(const embed_shape_t *shape, const void *weight, int64_t weight_stride, const void *ids,
               void *out, int64_t out_stride, hipStream_t stream)
{
    const int rc = check_embed(shape, weight, ids, out, false);
    if (rc != LIBSCAN_OK || shape->tokens == 0)
        return rc;
    EmbedRowsArgs a = {};
    a.weight = weight;
    a.out = out;
    a.ids = ids;
    a.weight_stride = weight_stride;
    a.out_stride = out_stride;
    a.dtype = shape->dtype;
    a.out_dtype = shape->out_dtype;
    a.id_bytes = shape->id_bytes;
    a.tokens = shape->tokens;
    a.rows = shape->rows;
    a.width = shape->width;
    a.scale = shape->scale;
    return hip_status(launch_embed_rows(a, stream));
}

size_t embed_grad_scratch_bytes(const embed_shape_t *shape)
{
    if (!shape || shape->tokens > EMBED_MAX_ROWS || shape->rows > EMBED_MAX_ROWS || shape->width > LIBSCAN_MAX_N)
        return with_header(0);
    return with_header(embed_grad_body_bytes(shape->tokens, shape->rows, shape->width));
}

int embed_grad(const embed_shape_t *shape, const void *dout, int64_t dout_stride, const void *ids,
               void *dweight, int64_t dweight_stride, int accumulate, void *scratch,
               size_t scratch_bytes, hipStream_t stream)
{
    const int rc = check_embed(shape, dweight, ids, dout, true);
    if (rc != LIBSCAN_OK)
        return rc;
    if ((accumulate & ~1) != 0)
        return LIBSCAN_ERR_ARG;
    const embed_shape_t &s = *shape;
    if (s.rows == 0 || (s.tokens == 0 && accumulate))
        return LIBSCAN_OK;
    if (!scratch)
        return LIBSCAN_ERR_NULL;
    Scratch scr;
    if (!carve(scratch, scratch_bytes, embed_grad_body_bytes(s.tokens, s.rows, s.width), &scr))
        return LIBSCAN_ERR_SCRATCH;
    EmbedGradArgs a = {};
    a.dout = dout;
    a.dweight = dweight;
    a.ids = ids;
    a.dout_stride = dout_stride;
    a.dweight_stride = dweight_stride;
    a.dtype = s.dtype;
    a.out_dtype = s.out_dtype;
    a.id_bytes = s.id_bytes;
    a.tokens = (uint32_t)s.tokens;
    a.rows = s.rows;
    a.width = s.width;
    a.scale = s.scale;
    a.accumulate = accumulate != 0;
    hipError_t e = prepare_state(scr, kKindData, 0, 0, 0, stream);
    if (e == hipSuccess)
        e = launch_embed_grad(a, scr.body(), stream);
    return hip_status(e);
}

int penalize_logits(const penalty_args_t *args, hipStream_t stream)
{
    if (!args)
        return LIBSCAN_ERR_NULL;
    const penalty_args_t &a = *args;
    if (bad_type(a.dtype))
        return LIBSCAN_ERR_ARG;
    const uint64_t most = LIBSCAN_MAX_N_INDEX;
    if (a.vocab > SAMPLE_MAX_VOCAB || a.rows > most || a.masks > most || a.past.count > most || a.bias.count > most)
        return LIBSCAN_ERR_SIZE;
    if ((uintptr_t)a.logits % element_bytes(a.dtype) != 0 || (uintptr_t)a.out % element_bytes(a.dtype) != 0 ||
        misaligned4(a.past.tokens) || misaligned4(a.past.ends) || misaligned4(a.prompts) ||
        misaligned4(a.repetitions) || misaligned4(a.presences) || misaligned4(a.frequencies) ||
        misaligned4(a.bias.tokens) || misaligned4(a.bias.ends) || misaligned4(a.bias_values) ||
        misaligned4(a.mask) || misaligned4(a.mask_slots))
        return LIBSCAN_ERR_ALIGN;
    if (a.rows == 0 || a.vocab == 0)
        return LIBSCAN_OK;
    if (!a.logits || !a.out || (a.past.count != 0 && !a.past.tokens) || (a.bias.count != 0 && !a.bias.tokens) ||
        (a.bias.tokens && a.bias.count != 0 && !a.bias_values) || (!a.mask && a.masks != 0))
        return LIBSCAN_ERR_NULL;
    if (a.logits == a.out && a.row_stride != a.out_stride)
        return LIBSCAN_ERR_ARG;
    return hip_status(launch_penalize(a, stream));
}

size_t sample_scratch_bytes(uint64_t rows, uint64_t vocab)
{
    if (rows > LIBSCAN_MAX_N_INDEX || vocab > SAMPLE_MAX_VOCAB)
        return with_header(0);
    return with_header(sample_body_bytes(rows, vocab));
}

int sample_logits(const sample_args_t *args, void *scratch, size_t scratch_bytes,
                  hipStream_t stream)
{
    if (!args)
        return LIBSCAN_ERR_NULL;
    const sample_args_t &a = *args;
    if (bad_type(a.dtype))
        return LIBSCAN_ERR_ARG;
    if (a.vocab > SAMPLE_MAX_VOCAB || a.rows > LIBSCAN_MAX_N_INDEX)
        return LIBSCAN_ERR_SIZE;
    if ((uintptr_t)a.logits % element_bytes(a.dtype) != 0 || misaligned4(a.u) ||
        misaligned4(a.temperatures) || misaligned4(a.top_ps) || misaligned4(a.min_ps) ||
        misaligned4(a.top_ks) || misaligned4(a.tokens) || misaligned4(a.logprobs) ||
        misaligned4(a.kept))
        return LIBSCAN_ERR_ALIGN;
    if (a.rows == 0)
        return LIBSCAN_OK;
    if ((!a.logits && a.vocab != 0) || !a.u || !a.tokens || !scratch)
        return LIBSCAN_ERR_NULL;
    Scratch s;
    if (!carve(scratch, scratch_bytes, sample_body_bytes(a.rows, a.vocab), &s))
        return LIBSCAN_ERR_SCRATCH;
    hipError_t e = prepare_state(s, kKindData, 0, 0, 0, stream);
    if (e == hipSuccess)
        e = launch_sample(a, s.body(), stream);
    return hip_status(e);
}

}  // extern "C"
