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
    DevError* err;
};

// One sequence: rows first .. first + n - 1 of the row tensors are its
// positions len - n .. len - 1.
struct Seq {
    int first, n, len;
};

// Sequence b; one whose rows do not lie in the row tensors is reported
// (info = b) and taken as having none.
__device__ __forceinline__ Seq load_seq(const View& v, int b) {
    Seq s;
    const int r0 = __ldg(v.row_start + b), r1 = __ldg(v.row_start + b + 1);
    s.first = r0;
    s.n = r1 - r0;
    s.len = __ldg(v.lens + b);
    if (r0 < 0 || r1 < r0 || r1 > v.n_rows || s.len < 0) {
        record_error(v.err, NVFP4_ERR_DEVICE, (uint32_t)b);
        s.n = 0;
        s.len = 0;
    }
    return s;
}

// The page that holds position pos of sequence b, or -1 (reported, info = b)
// when the table does not list one of the cache's pages for it.
__device__ __forceinline__ int page_of(const View& v, int b, int pos) {
    const int i = pos / v.page_size;
    const int p = i < v.max_pages ? __ldg(v.pages + (int64_t)b * v.max_pages + i) : -1;
    if (p >= 0 && p < v.n_pages) return p;
    record_error(v.err, NVFP4_ERR_DEVICE, (uint32_t)b);
    return -1;
}

// Row index of (page, head, position) in the cache's [..][head_dim] rows.
__device__ __forceinline__ int64_t cache_row(const View& v, int page, int head, int pos) {
    return ((int64_t)page * v.kv_heads + head) * v.page_size + pos % v.page_size;
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

// Whether the 16 keys from k0 on hold a key of the span (a page without one is
// not looked up: a sliding window's caller may have given it back).
__device__ __forceinline__ bool group_seen(const Span& s, int k0) {
    return k0 < s.hi && (k0 + kGroup > s.lo || k0 < s.sink_end);
}

// ---------------------------------------------------------------------------
// attention: what the kernel for few rows and the one for chunks share
// ---------------------------------------------------------------------------
constexpr float kLazy = 8.0f;     // a reference maximum moves when exceeded by more than 2^8
constexpr float kFloor = -1e30f;  // the reference before any visible key

struct AttnArgs {
    View v;
    const uint8_t* q;  // bf16 [n_rows][heads][d], ld_q elements between rows
    uint8_t* o;
    int64_t ld_q, ld_o;
    int heads, group, window, sinks, max_rows;
    int row_tiles, splits, split_tiles;
    float scale_log2;
    float* part_o;   // [splits][n_rows][heads][d]
    float2* part_ml; // [splits][n_rows][heads] (reference maximum, sum)
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

// Tiles of one split of a unit with `count` tiles.
__device__ __forceinline__ int tiles_per_split(const AttnArgs& a, int count) {
    return max(a.split_tiles, (count + a.splits - 1) / a.splits);
}

// The kernel for chunks (paged_attention.cu).
constexpr int kChunkRows = 256;  // (row, query head) pairs of a unit
constexpr int kChunkKeys = 128;
nvfp4_status launch_chunks(const AttnArgs& a, int64_t units, cudaStream_t stream);

}  // namespace paged
}  // namespace nvfp4
