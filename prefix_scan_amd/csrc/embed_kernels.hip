// embed_kernels.hip -- rows of a table by their ids, and the gradient of that
// (embed.hpp).
#include "embed.hpp"
#include "device_common.hpp"
#include "rows_io.hpp"

namespace libscan {

namespace {

// Eight elements of a row as floats, the first n of them.
template <class T>
__device__ __forceinline__ void load8(const T *at, int n, float (&f)[8])
{
    constexpr int V = kPiece<T>;
#pragma unroll
    for (int q = 0; q < 8 / V; ++q) {
        const piece_t r = load_piece<T>(at + q * V, n - q * V);
#pragma unroll
        for (int e = 0; e < V; ++e)
            f[q * V + e] = Unpack<T>::get(r, e);
    }
}

template <class T>
__device__ __forceinline__ void store8(T *at, int n, const float (&f)[8])
{
    constexpr int V = kPiece<T>;
#pragma unroll
    for (int q = 0; q < 8 / V; ++q) {
        float part[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            part[e] = f[q * V + e];
        store_piece<T>(at + q * V, Unpack<T>::pack(part), n - q * V);
    }
}

__device__ __forceinline__ int64_t id_at(const void *ids, int bytes, uint64_t i)
{
    return bytes == 8 ? static_cast<const int64_t *>(ids)[i] : (int64_t)static_cast<const int32_t *>(ids)[i];
}

// Lanes of a row and workgroups along it, of 8 elements each: the most lanes
// that leave few idle.
void row_lanes(uint64_t width, int *lanes, uint32_t *across)
{
    const uint64_t units = (width + 7) / 8;
    uint64_t least = ~0ull;
    for (int l = 256; l >= 8; l /= 2) {
        const uint64_t all = (units + l - 1) / l * l;
        if (all <= units + units / 8) {
            *lanes = l;
            *across = (uint32_t)(all / l);
            return;
        }
        if (all < least) {
            least = all;
            *lanes = l;
            *across = (uint32_t)(all / l);
        }
    }
}

constexpr int kRowsInFlight = 4;

// out[i] = scale weight[id i].  Bound: memory, the rows' bytes once in and once
// out; kRowsInFlight rows of a thread are under way at once.
template <class T, class O>
__global__ __launch_bounds__(256) void embed_rows_kernel(EmbedRowsArgs p)
{
    const int per = 256 / p.lanes;
    const uint64_t blocks = (p.tokens + per * kRowsInFlight - 1) / (per * kRowsInFlight) * p.across;
    for (uint64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const uint64_t c = ((b % p.across) * p.lanes + threadIdx.x % p.lanes) * 8;
        const uint64_t first = b / p.across * (per * kRowsInFlight) + threadIdx.x / p.lanes;
        if (c >= p.width)
            continue;
        const int n = p.width - c < 8 ? (int)(p.width - c) : 8;
        int64_t id[kRowsInFlight];
        float f[kRowsInFlight][8];
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
            const uint64_t r = first + (uint64_t)u * per;
            id[u] = r < p.tokens ? id_at(p.ids, p.id_bytes, r) : -1;
        }
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[u][e] = 0.f;
            if (id[u] >= 0 && (uint64_t)id[u] < p.rows)
                load8(static_cast<const T *>(p.weight) + id[u] * p.weight_stride + c, n, f[u]);
        }
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
            const uint64_t r = first + (uint64_t)u * per;
            if (r >= p.tokens)
                continue;
            const bool row = id[u] >= 0 && (uint64_t)id[u] < p.rows;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[u][e] = row ? f[u][e] * p.scale : 0.f;
            store8(static_cast<O *>(p.out) + (int64_t)r * p.out_stride + c, n, f[u]);
        }
    }
}

// --------------------------------------------------------------------------
// The sort: stable, by digits from the lowest, of (key, position)
// --------------------------------------------------------------------------

// Tiles whose keys each workgroup counts itself.  Whole calls (50021 x 64 bf16) with
// and without that, us: 2 tiles 36 and 53, 4 46 and 68, 8 62 and 85, 12 76 and 93,
// 16 92 and 98, 25 137 and 110.  (12 and 16 are not counted so all the same.)
constexpr uint32_t kFewTiles = 8;

// Parts of the table's gradient that the sort's kernels clear: each pass one,
// the counting before them, whose own work is short, the rest.
__device__ __forceinline__ int fill_parts(const EmbedGradArgs &p)
{
    return p.sort.tiles <= kFewTiles ? p.sort.passes : kSortMaxPasses + 1;
}

// A token's key: its row, or `rows` for an id that is no row, which comes last.
__device__ __forceinline__ uint32_t key_at(const EmbedGradArgs &p, uint32_t i)
{
    const int64_t id = id_at(p.ids, p.id_bytes, i);
    return id >= 0 && (uint64_t)id < p.rows ? (uint32_t)id : (uint32_t)p.rows;
}

// Zeros in the table's gradient, from the `from`-th of `parts` equal parts up to
// the `to`-th, by `count` workgroups of which this is number i.
template <class O>
__device__ void fill_rows(const EmbedGradArgs &p, int from, int to, int parts, uint32_t i, uint32_t count)
{
    const piece_t none = {0, 0, 0, 0};
    constexpr int V = kPiece<O>;
    const bool dense = p.dweight_stride == (int64_t)p.width;
    const uint64_t rows = dense ? 1 : p.rows, width = dense ? p.rows * p.width : p.width;
    const uint64_t units = (width + V - 1) / V, all = rows * units;
    const uint64_t lo = all / parts * from, hi = to == parts ? all : all / parts * to;
    for (uint64_t u = lo + (uint64_t)i * blockDim.x + threadIdx.x; u < hi; u += (uint64_t)count * blockDim.x) {
        const uint64_t r = dense ? 0 : u / units, c = (dense ? u : u % units) * V;
        O *const to = static_cast<O *>(p.dweight) + (int64_t)r * p.dweight_stride + c;
        if (width - c >= (uint64_t)V)
            store_piece_past(to, none);
        else
            store_piece<O>(to, none, (int)(width - c));
    }
}

// How many keys of each tile have each value of the first digit, and zeros
// where the later digits' are counted.
template <class O>
__global__ __launch_bounds__(kSortThreads) void embed_hist_kernel(EmbedGradArgs p)
{
    __shared__ uint32_t s_bin[kSortBins];
    if (blockIdx.x >= p.sort.tiles) {
        const int parts = fill_parts(p);
        fill_rows<O>(p, 0, parts - p.sort.passes, parts, blockIdx.x - p.sort.tiles, gridDim.x - p.sort.tiles);
        return;
    }
    const uint32_t tile = blockIdx.x, bins = 1u << p.sort.bits;
    for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads)
        s_bin[b] = 0;
    __syncthreads();
    const uint32_t lo = tile * kSortTile, hi = p.tokens - lo < kSortTile ? p.tokens : lo + kSortTile;
    for (uint32_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
        atomicAdd(&s_bin[key_at(p, i) & (bins - 1)], 1u);
    __syncthreads();
    for (uint32_t b = threadIdx.x; b < bins; b += kSortThreads) {
        p.hist[(uint64_t)tile * bins + b] = s_bin[b];
        for (int q = 1; q < p.sort.passes; ++q)
            p.hist[((uint64_t)q * p.sort.tiles + tile) * bins + b] = 0;
    }
}

// Each digit's counts become the sums over the tiles before; the whole to
// totals.  A workgroup has 64 digits, its 16 waves a part of the tiles each.
__global__ __launch_bounds__(1024) void embed_columns_kernel(uint32_t *hist, uint32_t *totals, uint32_t tiles,
                                                             uint32_t bins)
{
    __shared__ uint32_t s_sum[16][64];
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, b = blockIdx.x * 64 + lane;
    const uint32_t part = (tiles + 15) / 16, lo = wave * part, hi = lo + part < tiles ? lo + part : tiles;
    uint32_t sum = 0;
    if (b < bins)
        for (uint32_t t = lo; t < hi; ++t)
            sum += hist[(uint64_t)t * bins + b];
    s_sum[wave][lane] = sum;
    __syncthreads();
    uint32_t run = 0;
    for (uint32_t w = 0; w < wave; ++w)
        run += s_sum[w][lane];
    if (b >= bins)
        return;
    for (uint32_t t = lo; t < hi; ++t) {
        const uint32_t n = hist[(uint64_t)t * bins + b];
        hist[(uint64_t)t * bins + b] = run;
        run += n;
    }
    if (wave == 15)
        totals[b] = run;
}

// Exclusive sums of s_bin's kSortBins values, in place, by all threads.
__device__ __forceinline__ void scan_bins(uint32_t *s_bin, uint32_t *s_wave)
{
    static_assert(kSortThreads == kSortBins, "a thread a bin");
    const uint32_t x = s_bin[threadIdx.x], sum = wave_incl_add(x);
    if (threadIdx.x % 64 == 63)
        s_wave[threadIdx.x / 64] = sum;
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t w = 0; w < threadIdx.x / 64; ++w)
        before += s_wave[w];
    s_bin[threadIdx.x] = before + sum - x;
    __syncthreads();
}

struct SortShared {
    uint32_t bin[kSortBins];                              // counts, then where a digit's keys of the tile go
    uint32_t count[kSortThreads / 64][kSortBins];         // of each wave
    uint32_t before[kSortBins], others[kSortBins];        // of the tiles before, of all others (few tiles)
    uint32_t wave[kSortThreads / 64];
};

// One pass over one tile.  Each wave has a contiguous part of it, 64 keys at a
// time: lanes of one digit find each other by its bits, the lowest adds them
// up, and so a key's rank is the sum over the keys before it.  Of few tiles
// each counts the others' keys itself: counted for it by those that move them
// they cost an atomic each, which are served one after another from a line of
// memory (9001 keys: 12 us of the pass's 22).
__device__ void sort_tile(const EmbedGradArgs &p, SortShared &s, int pass, uint32_t tile)
{
    constexpr int kRounds = kSortTile / kSortThreads;
    const uint32_t bins = 1u << p.sort.bits, shift = pass * p.sort.bits, lane = threadIdx.x % 64,
                   wave = threadIdx.x / 64;
    const int from = (p.sort.passes - pass) & 1;          // the last pass writes [0]
    const uint32_t first = tile * kSortTile + wave * (kRounds * 64) + lane;
    uint32_t key[kRounds], at[kRounds], rank[kRounds];
    const bool few = p.sort.tiles <= kFewTiles;
    for (uint32_t w = 0; w < kSortThreads / 64; ++w)
        s.count[w][threadIdx.x] = 0;
    s.before[threadIdx.x] = s.others[threadIdx.x] = 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t i = first + r * 64;
        key[r] = 0;
        at[r] = i;
        if (i < p.tokens) {
            key[r] = pass == 0 ? key_at(p, i) : p.keys[from][i];
            if (pass != 0)
                at[r] = p.at[from][i];
        }
    }
    __syncthreads();
    for (uint32_t other = 0; few && other < p.sort.tiles; ++other) {
        if (other == tile)
            continue;
        uint32_t k[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const uint32_t i = other * kSortTile + r * kSortThreads + threadIdx.x;
            k[r] = i >= p.tokens ? 0 : pass == 0 ? key_at(p, i) : p.keys[from][i];
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (other * kSortTile + r * kSortThreads + threadIdx.x < p.tokens)
                atomicAdd(&(other < tile ? s.before : s.others)[k[r] >> shift & (bins - 1)], 1u);
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const bool in = first + r * 64 < p.tokens;
        const uint32_t d = key[r] >> shift & (bins - 1);
        uint64_t same = ballot(in);
        for (int b = 0; b < p.sort.bits; ++b) {
            const uint64_t set = ballot((d >> b & 1) != 0);
            same &= (d >> b & 1) ? set : ~set;
        }
        volatile uint32_t *const count = &s.count[wave][d];
        const uint32_t before = *count;
        rank[r] = before + __popcll(same & lanemask_lt());
        __builtin_amdgcn_wave_barrier();
        if (in && (same & lanemask_lt()) == 0)
            *count = before + __popcll(same);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    // Digit `threadIdx.x`: where its keys of this tile start.
    {
        const uint32_t b = threadIdx.x;
        uint32_t all = 0, before = 0;
        if (few) {
            before = s.before[b];
            all = before + s.others[b];
            for (int w = 0; w < kSortThreads / 64; ++w)
                all += s.count[w][b];
        } else if (b < bins) {
            const uint32_t *const hist = p.hist + (uint64_t)pass * p.sort.tiles * bins;
            if (p.totals) {
                before = hist[(uint64_t)tile * bins + b];
                all = p.totals[b];
            } else {
                for (uint32_t t = 0; t < p.sort.tiles; ++t) {
                    const uint32_t n = hist[(uint64_t)t * bins + b];
                    all += n;
                    before += t < tile ? n : 0;
                }
            }
        }
        s.bin[b] = all;
        __syncthreads();
        scan_bins(s.bin, s.wave);
        uint32_t run = s.bin[b] + before;
        for (int w = 0; w < kSortThreads / 64; ++w) {
            const uint32_t n = s.count[w][b];
            s.count[w][b] = run;
            run += n;
        }
    }
    __syncthreads();
    uint32_t *const next = p.hist + (uint64_t)(pass + 1) * p.sort.tiles * bins;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (first + r * 64 >= p.tokens)
            continue;
        const uint32_t to = s.count[wave][key[r] >> shift & (bins - 1)] + rank[r];
        p.keys[from ^ 1][to] = key[r];
        p.at[from ^ 1][to] = at[r];
        if (!few && pass + 1 < p.sort.passes)
            atomicAdd(&next[(uint64_t)(to / kSortTile) * bins + (key[r] >> (shift + p.sort.bits) & (bins - 1))], 1u);
    }
}

template <class O>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(EmbedGradArgs p, int pass)
{
    __shared__ SortShared s;
    if (blockIdx.x >= p.sort.tiles) {
        const int parts = fill_parts(p), part = parts - p.sort.passes + pass;
        fill_rows<O>(p, part, part + 1, parts, blockIdx.x - p.sort.tiles, gridDim.x - p.sort.tiles);
    } else {
        sort_tile(p, s, pass, blockIdx.x);
    }
}

// All passes over a list of one tile.
template <class O>
__global__ __launch_bounds__(kSortThreads) void embed_sort_one_kernel(EmbedGradArgs p)
{
    __shared__ SortShared s;
    if (blockIdx.x != 0) {
        fill_rows<O>(p, 0, 1, 1, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    for (int pass = 0; pass < p.sort.passes; ++pass) {
        sort_tile(p, s, pass, 0);
        __threadfence_block();
        __syncthreads();
    }
}

// --------------------------------------------------------------------------
// Sums of the sorted list's rows
// --------------------------------------------------------------------------

constexpr int kSumBatch = 16;

// N elements of a row, the first n of them.
template <int N, class O>
__device__ __forceinline__ void load_some(const O *at, int n, float (&f)[N])
{
    if constexpr (N == 8) {
        load8(at, n, f);
    } else {
        const Four<O> x = load_four(at, n);
#pragma unroll
        for (int e = 0; e < N; ++e)
            f[e] = x.get(e);
    }
}
template <int N, class O>
__device__ __forceinline__ void store_some(O *at, int n, const float (&f)[N])
{
    if constexpr (N == 8)
        store8(at, n, f);
    else
        store_four(at, Four<O>::of(f), n);
}

template <class O, int N>
__device__ __forceinline__ void put_row(const EmbedGradArgs &p, uint32_t row, uint64_t c, int n, float (&sum)[N])
{
    O *const at = static_cast<O *>(p.dweight) + (int64_t)row * p.dweight_stride + c;
    float old[N];
    if (p.accumulate)
        load_some<N>(at, n, old);
#pragma unroll
    for (int e = 0; e < N; ++e)
        sum[e] = p.accumulate ? __builtin_fmaf(p.scale, sum[e], old[e]) : p.scale * sum[e];
    store_some<N>(at, n, sum);
}

// One chunk of the sorted list, 64 pieces of its rows, by a wave: runs that lie
// within it are done, what it holds of others goes to its partial rows -- 0 of
// the run that comes from the chunks before, 1 of the one that starts here and
// goes on.
// Bound: memory, the rows' bytes.  The rows of kSumBatch entries are under way
// at once, and a chunk is as few entries where that leaves waves enough: keys
// are the same in all lanes, so that a run's end costs a scalar branch.
template <class T, class O, bool WHOLE>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedGradArgs p)
{
    constexpr int V = kPiece<T>;
    const uint32_t lane = threadIdx.x % 64;
    const uint64_t waves = (uint64_t)p.chunks * p.across;
    for (uint64_t w = (uint64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64); w < waves;
         w += (uint64_t)gridDim.x * 4) {
        const uint32_t chunk = (uint32_t)(w / p.across);
        const uint64_t c = ((w % p.across) * 64 + lane) * V;
        const int n = c >= p.width ? 0 : p.width - c < (uint64_t)V ? (int)(p.width - c) : V;
        const uint32_t lo = chunk * p.chunk, hi = p.tokens - lo < p.chunk ? p.tokens : lo + p.chunk;
        const auto entry = [&](uint32_t i0) { return i0 + lane < hi ? i0 + lane : hi - 1; };
        uint32_t keys = p.keys[0][entry(lo)], ats = p.at[0][entry(lo)];
        const uint32_t before = lo ? p.keys[0][lo - 1] : ~0u, after = hi < p.tokens ? p.keys[0][hi] : ~0u;
        uint32_t cur = __builtin_amdgcn_readfirstlane(keys);
        bool started = before != cur;
        float sum[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            sum[e] = 0.f;
        const auto flush = [&](bool ended) {
            if (cur >= p.rows || n == 0)
                return;
            const int m = WHOLE ? V : n;
            if (started && ended) {
                put_row<O>(p, cur, c, m, sum);
            } else {
                float *const to = p.partial + ((uint64_t)chunk * 2 + (started ? 1 : 0)) * p.width + c;
                store_some<V>(to, m, sum);
            }
        };
        for (uint32_t i0 = lo; i0 < hi; i0 += kSumBatch) {
            const uint32_t keys_now = keys, ats_now = ats;
            if (i0 + kSumBatch < hi) {
                keys = p.keys[0][entry(i0 + kSumBatch)];
                ats = p.at[0][entry(i0 + kSumBatch)];
            }
            uint32_t key[kSumBatch];
            piece_t raw[kSumBatch];
#pragma unroll
            for (int u = 0; u < kSumBatch; ++u) {
                key[u] = __builtin_amdgcn_readlane(keys_now, u);
                const uint32_t at = __builtin_amdgcn_readlane(ats_now, u);
                raw[u] = piece_t{0, 0, 0, 0};
                if (i0 + u < hi && key[u] < p.rows && (!WHOLE || n != 0))
                    raw[u] = load_piece<T>(static_cast<const T *>(p.dout) + (int64_t)at * p.dout_stride + c,
                                           WHOLE ? V : n);
            }
#pragma unroll
            for (int u = 0; u < kSumBatch; ++u) {
                if (i0 + u >= hi)
                    continue;
                if (key[u] != cur) {
                    flush(true);
                    cur = key[u];
                    started = true;
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        sum[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < V; ++e)
                    sum[e] += Unpack<T>::get(raw[u], e);
            }
        }
        flush(after != cur);
    }
}

// The runs that chunks share: where one starts, its partial rows are added, in
// eight parts one after another and these in their order.  A workgroup looks at
// kJoinChunks chunks, 256 columns of their rows.
constexpr int kJoinChunks = 4;

template <class O>
__global__ __launch_bounds__(256) void embed_join_kernel(EmbedGradArgs p)
{
    __shared__ float s_sum[8][256];
    const uint32_t across = (uint32_t)((p.width + 255) / 256), lane = threadIdx.x % 64;
    const uint64_t blocks = (uint64_t)((p.chunks + kJoinChunks - 1) / kJoinChunks) * across;
    for (uint64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const uint32_t chunk0 = (uint32_t)(b / across) * kJoinChunks, mine = chunk0 + lane;
        uint32_t keys = 0;
        bool shared = false;
        if (lane < kJoinChunks && mine + 1 < p.chunks) {
            const uint32_t lo = mine * p.chunk, hi = lo + p.chunk;
            const uint32_t after = p.keys[0][hi], from = p.keys[0][lo], before = lo ? p.keys[0][lo - 1] : ~0u;
            keys = p.keys[0][hi - 1];
            shared = keys < p.rows && after == keys && (from != keys || before != keys);
        }
        // The same in all waves.
        for (uint64_t left = __ballot(shared); left != 0; left &= left - 1) {
            const uint32_t which = (uint32_t)__builtin_ctzll(left), chunk = chunk0 + which;
            const uint32_t key = __builtin_amdgcn_readlane(keys, which);
            // The last chunk that begins with the key: among the next 64, or by
            // steps of a 64th of what is left.
            uint32_t last = chunk + 1, past = p.chunks;
            for (uint32_t step = 1; past - last > 1; step = (past - last + 63) / 64) {
                const uint64_t at = last + (uint64_t)(lane + 1) * step;
                const uint64_t same = __ballot(at < past && p.keys[0][(at < past ? at : last) * p.chunk] == key);
                const uint32_t more = (uint32_t)__popcll(same) * step;
                last += more;
                past = more == 64 * step || past - last < step ? past : last + step;
            }
            const uint64_t c = (b % across) * 256 + threadIdx.x % 32 * 8;
            const int n = c < p.width ? (p.width - c < 8 ? (int)(p.width - c) : 8) : 0;
            const uint32_t part = threadIdx.x / 32, many = last - chunk + 1, each = (many + 7) / 8;
            float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (uint32_t i = part * each; i < many && i < (part + 1) * each && n > 0; ++i) {
                float f[8];
                load8(p.partial + ((uint64_t)(chunk + i) * 2 + (i == 0 ? 1 : 0)) * p.width + c, n, f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] += f[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s_sum[part][threadIdx.x % 32 * 8 + e] = sum[e];
            __syncthreads();
            if (part == 0 && n > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    for (int i = 1; i < 8; ++i)
                        sum[e] += s_sum[i][threadIdx.x * 8 + e];
                put_row<O>(p, key, c, n, sum);
            }
            __syncthreads();
        }
    }
}

template <class T>
hipError_t rows_from(const EmbedRowsArgs &a, unsigned grid, hipStream_t stream)
{
    switch (a.out_dtype) {
    case LIBSCAN_F32: embed_rows_kernel<T, float><<<grid, 256, 0, stream>>>(a); break;
    case LIBSCAN_BF16: embed_rows_kernel<T, __bf16><<<grid, 256, 0, stream>>>(a); break;
    default: embed_rows_kernel<T, _Float16><<<grid, 256, 0, stream>>>(a); break;
    }
    return hipGetLastError();
}

// Workgroups of a loop over `blocks`: a grid holds fewer than 2^32 threads.
unsigned grid_of(uint64_t blocks) { return (unsigned)(blocks < (1u << 22) ? blocks : 1u << 22); }

// Rows of whole pieces have a kernel of their own, a third as long, without the
// cut ones' loads and stores.  Whole calls with it and without, us: 500 rows of 520
// 24.7 and 25.9, 9001 52.8 and 54.5, 32768 f32 rows of 1024 103.0 and 105.3, 65536
// bf16 ones 136.3 and 136.9.
template <class T, class O>
void sum_from(const EmbedGradArgs &a, unsigned grid, hipStream_t stream)
{
    if (a.width % kPiece<T> == 0)
        embed_sum_kernel<T, O, true><<<grid, 256, 0, stream>>>(a);
    else
        embed_sum_kernel<T, O, false><<<grid, 256, 0, stream>>>(a);
}

template <class O>
hipError_t grad_to(const EmbedGradArgs &a, hipStream_t stream)
{
    // What else a kernel of the sort does: zeros in its part of the table.
    const unsigned fill = a.accumulate ? 0 : 1024;
    if (a.sort.tiles == 1) {
        embed_sort_one_kernel<O><<<1 + fill, kSortThreads, 0, stream>>>(a);
    } else {
        const uint32_t bins = 1u << a.sort.bits;
        if (a.sort.tiles > kFewTiles)
            embed_hist_kernel<O><<<a.sort.tiles + fill, kSortThreads, 0, stream>>>(a);
        for (int pass = 0; pass < a.sort.passes; ++pass) {
            if (a.totals)
                embed_columns_kernel<<<(bins + 63) / 64, 1024, 0, stream>>>(
                    a.hist + (uint64_t)pass * a.sort.tiles * bins, a.totals, a.sort.tiles, bins);
            embed_sort_kernel<O><<<a.sort.tiles + fill, kSortThreads, 0, stream>>>(a, pass);
        }
    }
    if (a.tokens == 0)
        return hipGetLastError();
    const unsigned grid = grid_of(((uint64_t)a.chunks * a.across + 3) / 4);
    switch (a.dtype) {
    case LIBSCAN_F32: sum_from<float, O>(a, grid, stream); break;
    case LIBSCAN_BF16: sum_from<__bf16, O>(a, grid, stream); break;
    default: sum_from<_Float16, O>(a, grid, stream); break;
    }
    if (a.chunks > 1)
        embed_join_kernel<O><<<grid_of((uint64_t)((a.chunks + kJoinChunks - 1) / kJoinChunks) *
                                       ((a.width + 255) / 256)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

// Tiles whose counts each workgroup adds up by itself, without a kernel between the
// passes that does.  Whole calls (50021 x 8 bf16) without that kernel and with it,
// us: 16 tiles 96 and 95, 32 112 and 104, 64 142 and 121, 128 188 and 141, 192 239 and
// 163, 512 553 and 334: it would be no loss from 16 tiles on.
constexpr uint32_t kSomeTiles = 128;

size_t up(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

SortPlan sort_plan(uint64_t tokens, uint64_t rows)
{
    int bits = 1;
    while (bits < 32 && (rows >> bits) != 0)      // keys are 0 .. rows
        ++bits;
    SortPlan s;
    s.passes = (bits + kSortBits - 1) / kSortBits;
    s.bits = (bits + s.passes - 1) / s.passes;
    s.tiles = (uint32_t)((tokens + kSortTile - 1) / kSortTile);
    return s;
}

// As few as leave some 2048 chunks: a chunk is a wave's work from its first entry to
// its last, and each leaves up to two rows to be joined.  Added to a table of 20011
// rows (bf16), us by chunks of 16, 32, 64 and 128 entries:
//      9001 tokens of 520    44   50   62   87
//     65536                 122  115  120  143
//    262144                 268  214  190  183
//     16384 of 2048          68   72   82  110
//    131072                 316  284  268  266
uint32_t embed_chunk(uint64_t tokens)
{
    uint32_t e = kSumBatch;
    while (e < 128 && tokens / e > 2048)
        e *= 2;
    return e;
}

size_t embed_grad_body_bytes(uint64_t tokens, uint64_t rows, uint64_t width)
{
    const SortPlan s = sort_plan(tokens, rows);
    const uint64_t chunks = (tokens + embed_chunk(tokens) - 1) / embed_chunk(tokens);
    return 4 * up(tokens * 4) + up(((uint64_t)s.passes * s.tiles + 1) << s.bits << 2) + up(chunks * 2 * width * 4);
}

hipError_t launch_embed_rows(EmbedRowsArgs a, hipStream_t stream)
{
    row_lanes(a.width, &a.lanes, &a.across);
    const uint64_t per = (uint64_t)(256 / a.lanes) * kRowsInFlight;
    const unsigned grid = grid_of((a.tokens + per - 1) / per * a.across);
    switch (a.dtype) {
    case LIBSCAN_F32: return rows_from<float>(a, grid, stream);
    case LIBSCAN_BF16: return rows_from<__bf16>(a, grid, stream);
    default: return rows_from<_Float16>(a, grid, stream);
    }
}

hipError_t launch_embed_grad(EmbedGradArgs a, void *body, hipStream_t stream)
{
    a.sort = sort_plan(a.tokens, a.rows);
    a.chunk = embed_chunk(a.tokens);
    a.chunks = (a.tokens + a.chunk - 1) / a.chunk;
    const uint64_t piece = 64 * (a.dtype == LIBSCAN_F32 ? 4 : 8);
    a.across = (uint32_t)((a.width + piece - 1) / piece);
    uint8_t *at = static_cast<uint8_t *>(body);
    const auto take = [&](size_t bytes) {
        void *p = at;
        at += up(bytes);
        return p;
    };
    for (int i = 0; i < 2; ++i) {
        a.keys[i] = static_cast<uint32_t *>(take((size_t)a.tokens * 4));
        a.at[i] = static_cast<uint32_t *>(take((size_t)a.tokens * 4));
    }
    const uint64_t cells = ((uint64_t)a.sort.passes * a.sort.tiles) << a.sort.bits;
    a.hist = static_cast<uint32_t *>(take((cells + (1ull << a.sort.bits)) * 4));
    a.totals = a.sort.tiles > kSomeTiles ? a.hist + cells : nullptr;
    a.partial = static_cast<float *>(take(0));
    switch (a.out_dtype) {
    case LIBSCAN_F32: return grad_to<float>(a, stream);
    case LIBSCAN_BF16: return grad_to<__bf16>(a, stream);
    default: return grad_to<_Float16>(a, stream);
    }
}

}  // namespace libscan
