// paged.cuh -- what the kernels over the paged NVFP4 cache share: the sequences
// of a step, where a position lies, and which keys a row sees.
#pragma once

#include "common.cuh"

namespace nvfp4 {
namespace paged {

constexpr int kGroup = 16;  // keys that always lie in one page (page_size is a multiple)

// The cache and the step's sequences as a kernel sees them (t = 0: K, 1: V).
struct View {
    const uint8_t* codes[2];   // [n_pages][kv_heads][page_size][head_dim / 2]
    const uint8_t* scales[2];  // [n_pages][kv_heads][page_size][head_dim / 16]
    const float* a32[2];
    const int32_t* row_start;
    const int32_t* lens;
    const int32_t* pages;
    int n_pages, page_size, kv_heads, d;
    int page_shift;  // page_size = 2^page_shift, or -1
    int n_seqs, max_pages, n_rows;
    int room;  // positions that a page table has room for (at most 2^30)
    DevError* err;
};

// One sequence: rows first .. first + n - 1 of the row tensors are its
// positions len - n .. len - 1.
struct Seq {
    int first, n, len;
};

// Sequence b; one whose rows do not lie in the row tensors, or whose length not
// in the page table, is reported (info = b) and taken as having none: whatever
// the arrays hold, a launch's work is bounded and no position overflows.
__device__ __forceinline__ Seq load_seq(const View& v, int b) {
    Seq s;
    const int r0 = ld_coherent(v.row_start + b), r1 = ld_coherent(v.row_start + b + 1);
    s.first = r0;
    s.n = r1 - r0;
    s.len = ld_coherent(v.lens + b);
    if (r0 < 0 || r1 < r0 || r1 > v.n_rows || s.len < 0 || s.len > v.room) {
        record_error(v.err, NVFP4_ERR_DEVICE, (uint32_t)b);
        s.n = 0;
        s.len = 0;
    }
    return s;
}

// The page that holds position pos < len of sequence b, or -1 (reported, info =
// b) when the table does not list one of the cache's pages for it.
__device__ __forceinline__ int page_of(const View& v, int b, int pos) {
    const int p = ld_coherent(v.pages + (int64_t)b * v.max_pages + pos / v.page_size);
    if (p >= 0 && p < v.n_pages) return p;
    record_error(v.err, NVFP4_ERR_DEVICE, (uint32_t)b);
    return -1;
}

// Entry i of a sequence's page table for the attention, in which -1 stands for
// a page that is not needed: an entry below 0 becomes -2.
__device__ __forceinline__ int listed(const int32_t* table, int i) {
    const int p = ld_coherent(table + i);
    return p < 0 ? -2 : p;
}

// The keys that some position of [p0, p1] sees, as two ranges [0, sink_end)
// and [lo, p1]; sink_end <= lo.  Position p sees j <= p with j > p - window or
// j < sinks (window 0: every j <= p).
struct Span {
    int sink_end, lo, hi;  // [0, sink_end) and [lo, hi)
};

__host__ __device__ __forceinline__ Span visible_span(int p0, int p1, int window, int sinks) {
    Span s;
    s.hi = p1 + 1 > 0 ? p1 + 1 : 0;
    s.lo = window > 0 && p0 - window + 1 > 0 ? p0 - window + 1 : 0;
    if (s.lo > s.hi) s.lo = s.hi;
    s.sink_end = window > 0 ? (sinks < s.lo ? sinks : s.lo) : 0;
    return s;
}

// The tiles of T keys that hold a key of the span, numbered 0 .. count - 1:
// first those of the sinks, then those of [lo, hi) that are not among them.
template <int T>
struct Tiles {
    int n_sink, first, count;
    __host__ __device__ __forceinline__ explicit Tiles(const Span& s) {
        n_sink = (s.sink_end + T - 1) / T;
        first = s.lo / T;
        if (first < n_sink) first = n_sink;
        const int end = (s.hi + T - 1) / T;
        count = n_sink + (end > first ? end - first : 0);
    }
    __host__ __device__ __forceinline__ int key0(int i) const { return (i < n_sink ? i : first + i - n_sink) * T; }
};

// Whether the 16 keys from k0 on hold a key of the span.  (A page without one is
// not looked up: a sliding window's caller may have given it back.  Places of a
// page that no row sees may hold anything, a NaN scale too.)
__device__ __forceinline__ bool group_seen(const Span& s, int k0) {
    return k0 < s.hi && (k0 + kGroup > s.lo || k0 < s.sink_end);
}

// ---------------------------------------------------------------------------
// attention: what the kernel for few rows and the one for chunks share
// ---------------------------------------------------------------------------
// The kernel for chunks (paged_attention.cu).
constexpr int kChunkRows = 256;  // (row, query head) pairs of a unit
constexpr int kChunkKeys = 64;
constexpr int kChunkCtas = 148;  // one an SM
constexpr int kChunkLeast = 3;   // tiles of a run (16 rows over 1000 keys: 17.3 us with 3, 19.4 with 4)
struct AttnArgs;
nvfp4_status launch_chunks(const AttnArgs& a, unsigned ctas, cudaStream_t stream);

// A row's weights are taken relative to a reference that is set kHead binary
// orders below the largest score so far and moves when that is exceeded by more
// than kLazy orders (decode; chunks: when a tile's weights sum above 2^15).  So
// the weights reach 2^15 at most, which binary16 holds, and keep its 11 bits down
// to 2^-21 of the largest and 2^-32 of it below: with the reference at the
// largest score itself, thousands of keys 24 to 26 orders below an attention
// sink lost their part of the result or doubled it.
constexpr float kLazy = 8.0f, kHead = 7.0f;
constexpr float kFloor = -1e30f;  // the reference before any visible key

struct AttnArgs {
    View v;
    const uint8_t* q;  // bf16 [n_rows][heads][d], ld_q elements between rows
    uint8_t* o;
    int64_t ld_q, ld_o;
    int group, window, sinks, max_rows;
    int row_tiles;  // units of the most rows a sequence may have
    float scale_log2;
    int4* cut;        // [workers]: (pieces of the unit that it begins and does not end, or 0; its pair, head, rows)
    float* part_o;    // [workers][2][cols][d] unnormalised
    float2* part_ml;  // [workers][2][cols] (reference maximum, sum)
};

// Rows f0 .. f0 + cols - 1 of a sequence's n * group (row, query head) pairs.
struct Rows {
    int n;     // pairs in the unit
    Span span;
};

__device__ __forceinline__ Rows unit_rows(const AttnArgs& a, const Seq& s, int f0, int cols) {
    Rows r;
    r.n = min(cols, s.n * a.group - f0);
    if (r.n <= 0) {
        r.n = 0;
        r.span = Span{0, 0, 0};
        return r;
    }
    const int p = s.len - s.n;
    r.span = visible_span(p + f0 / a.group, p + (f0 + r.n - 1) / a.group, a.window, a.sinks);
    return r;
}

// The work of a launch is one list of key tiles: for every pair of a sequence
// and a run of its rows, for every K/V head, that unit's tiles.  The list is
// cut into equal runs, one a worker (a warp of the decode kernel, a CTA of the
// chunk kernel), whatever the lengths; a unit that lies in several runs leaves
// a piece in each, which combine_kernel joins.  Worker k keeps the piece of a
// unit that began before its run at 2 k, of one that ends after it at 2 k + 1.
struct Piece {
    int b, head, f0;   // sequence, K/V head, first (row, query head) pair
    int begin, end;    // tiles of the unit (a unit that sees none has one empty piece: 0, 0)
    int slot;          // where the piece is kept, or -1 when it is the whole unit
    int pair, pieces;  // of a unit that begins here and ends in a later run: its pieces
    Seq s;
    Rows rows;
};

struct Run {
    int64_t x, end, base;  // the run's next tile and end, first tile of the pair
    int64_t per;           // tiles of every run but the last
    int worker, pair;
};

// What beginning and ending a unit costs, in tiles: a unit counts as that many
// more, so that runs of short units are no longer than the others.  (Chunks, 6
// sequences of up to 700 rows x 32 heads over 8: 193 us with 1, 184 with 4, 169
// with 8, 172 with 14; decode steps differ by 2 us between 3 and 8.)
template <int COLS>
constexpr int kUnitCost = COLS == kChunkRows ? 8 : 5;

// Tiles of pair j as counted in the list (0: no rows), and as they are.
template <int COLS, int T>
__device__ __forceinline__ int pair_tiles(const AttnArgs& a, int j, Seq* seq, Rows* rows, int* real) {
    const int b = j / a.row_tiles;
    *seq = load_seq(a.v, b);
    if (seq->n > a.max_rows) {  // more rows than the launch was sized for
        record_error(a.v.err, NVFP4_ERR_DEVICE, (uint32_t)b);
        seq->n = 0;
    }
    *rows = unit_rows(a, *seq, j % a.row_tiles * COLS, COLS);
    if (rows->n == 0) return 0;
    const Tiles<T> tiles(rows->span);
    *real = tiles.count;
    return tiles.count + kUnitCost<COLS>;
}

template <int THREADS>
struct RunScratch {
    long long warp_sum[THREADS / 32];
    long long first[THREADS];  // first tile of each thread's pairs
};

// The run of worker blockIdx.x * WORKERS + worker (all THREADS threads; no run
// is shorter than `least` tiles).
template <int COLS, int T, int THREADS, int WORKERS>
__device__ __forceinline__ Run make_run(const AttnArgs& a, int worker, int least, RunScratch<THREADS>& sh) {
    const int pairs = a.v.n_seqs * a.row_tiles, each = (pairs + THREADS - 1) / THREADS;
    const int j0 = min(pairs, (int)threadIdx.x * each), j1 = min(pairs, j0 + each);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Seq s;
    Rows r;
    int real;
    long long sum = 0;
    for (int j = j0; j < j1; j++) sum += pair_tiles<COLS, T>(a, j, &s, &r, &real);
    sum *= a.v.kv_heads;
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; w++) {
        if (w < warp) before += sh.warp_sum[w];
        total += sh.warp_sum[w];
    }
    sh.first[threadIdx.x] = before + incl - sum;
    __syncthreads();
    const long long workers = (long long)gridDim.x * WORKERS;
    Run run;
    run.worker = (int)blockIdx.x * WORKERS + worker;
    run.per = max((long long)least, (total + workers - 1) / workers);
    run.x = run.worker * run.per;
    run.end = min((int64_t)total, run.x + run.per);
    run.pair = pairs;
    run.base = 0;
    if (run.x >= run.end) return run;
    // the last thread whose pairs begin at or before the run, then the pair among them
    int lo = 0, hi = THREADS;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (sh.first[mid] <= run.x) lo = mid;
        else hi = mid;
    }
    run.pair = lo * each;
    run.base = sh.first[lo];
    return run;  // (next_piece walks on from there)
}

// The run's next piece; false at its end.
template <int COLS, int T>
__device__ __forceinline__ bool next_piece(const AttnArgs& a, Run& run, Piece& p) {
    while (run.x < run.end && run.pair < a.v.n_seqs * a.row_tiles) {
        int real = 0;
        const int n = pair_tiles<COLS, T>(a, run.pair, &p.s, &p.rows, &real);
        const int64_t all = (int64_t)n * a.v.kv_heads;
        if (run.x >= run.base + all) {
            run.base += all;
            run.pair++;
            continue;
        }
        const int64_t off = run.x - run.base;
        p.b = run.pair / a.row_tiles;
        p.f0 = run.pair % a.row_tiles * COLS;
        p.head = (int)(off / n);
        p.begin = (int)(off % n);
        p.end = (int)min((int64_t)n, p.begin + (run.end - run.x));
        run.x += p.end - p.begin;
        if (p.begin >= real && p.begin > 0) continue;  // the unit's cost alone is left
        p.end = min(p.end, real);
        p.pair = run.pair;
        p.pieces = 0;
        if (p.begin > 0) {
            p.slot = 2 * run.worker;
        } else if (p.end < real) {
            p.slot = 2 * run.worker + 1;
            p.pieces = (int)(1 + (real - p.end + run.per - 1) / run.per);
        } else {
            p.slot = -1;
        }
        return true;
    }
    return false;
}

}  // namespace paged
}  // namespace nvfp4
