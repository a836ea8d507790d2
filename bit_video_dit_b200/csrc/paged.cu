// The paged NVFP4 cache: token rows quantized into pages as they are written,
// read back to bf16, and attention of few rows (a decode step's) over it.  The
// reading note's KV store (section 二 推理底座) quantizes a whole frame-chunk with
// the chunk's own tensor scale; here a sequence grows by any number of tokens
// a step, so the tensor scale is the cache's, given once (delayed scaling), and
// the E4M3 block scales follow each token.
//
// Layout: page p, K/V head h, token o of the page: row (p * kv_heads + h) *
// page_size + o of head_dim elements.  One head's tokens of a page are
// contiguous, so an attention tile of one head reads whole lines.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fp4mma.cuh"
#include "paged.cuh"

namespace nvfp4 {
namespace paged {

using namespace fp4mma;

// ---------------------------------------------------------------------------
// append and gather.  Memory bound: 2 bytes an element one way, 9/16 the other.
// A lane holds one 16-element block, so a warp has the head_dim / 16 blocks of
// 4 (head_dim 128) or 8 (64) consecutive rows of one head: it reads and writes
// whole 32-byte sectors on both sides (read and write in one access a lane where
// the rows are aligned to that: 53 -> 37 us for 51k rows of 8 heads of 64 read
// back).  Finding a row's place takes five dependent loads, so a warp takes
// several heads of K and V of its rows, 4 (append, whose arithmetic needs the
// registers) or 8 (gather) of them at a time.  2640 rows x 24 heads x 128 (calls
// in a graph, data from DRAM): append with RoPE 14.1 us (3.0 TB/s), gather 10.9
// (3.8); the 51k rows 35.2 (4.8).
// ---------------------------------------------------------------------------
constexpr int kRowWarps = 8;

struct RowArgs {
    View v;
    uint8_t* rows[2];  // bf16 K, V rows [n_rows][kv_heads][d]
    int64_t ld[2];     // elements between rows
    const float* rope_cos;  // [n_rows][d / 2] or NULL
    const float* rope_sin;
    int items, parts;  // (head, K or V) pairs, warps that share them
    bool wide;         // every block of the rows lies on 32 bytes
};

// A block's 32 bytes: in one access where they are aligned to that (two of 16
// bytes each leave half a sector to the other instruction).
__device__ __forceinline__ void load32(const uint8_t* p, bool wide, uint4* x) {
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x[0].x), "=r"(x[0].y), "=r"(x[0].z), "=r"(x[0].w), "=r"(x[1].x), "=r"(x[1].y), "=r"(x[1].z),
                       "=r"(x[1].w)
                     : "l"(p)
                     : "memory");
    } else {
        x[0] = ld_coherent(reinterpret_cast<const uint4*>(p));
        x[1] = ld_coherent(reinterpret_cast<const uint4*>(p) + 1);
    }
}
__device__ __forceinline__ void store32(uint8_t* p, bool wide, const uint32_t* o) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                     "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// The last sequence b with row_start[b] <= row (the warp searches together,
// 32 entries at a time).
__device__ __forceinline__ int find_seq(const View& v, int row, int lane) {
    int lo = 0, hi = v.n_seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t i = lo + (int64_t)lane * step;
        const bool le = lane == 0 || (i < hi && ld_coherent(v.row_start + i) <= row);
        lo += (__popc(__ballot_sync(0xFFFFFFFFu, le)) - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// A lane's block of one (head, K or V) item on its way.
struct RowBlock {
    uint4 x[2];  // append: 16 bf16; gather: .x[0].x, .y the codes, .z the scale
};

// 16 elements (K with RoPE when tables are given, as nvfp4_kv_append_rope) to
// codes and scale at cache row `at`, block `blk`.
__device__ __forceinline__ void append_block(const RowArgs& a, const RowBlock& r, int t, float a32, int row, int blk,
                                             uint32_t at) {
    const View& v = a.v;
    float x[16];
    bf16x8_to_f32(r.x[0], x);
    bf16x8_to_f32(r.x[1], x + 8);
    if (t == 0 && a.rope_cos) {
        const int64_t off = (int64_t)row * (v.d / 2) + 8 * blk;
        const float4* pc = reinterpret_cast<const float4*>(a.rope_cos + off);
        const float4* ps = reinterpret_cast<const float4*>(a.rope_sin + off);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float4 c4 = ld_coherent(pc + i), s4 = ld_coherent(ps + i);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float &x0 = x[8 * i + 2 * e], &x1 = x[8 * i + 2 * e + 1];
                const float y0 = __fsub_rn(__fmul_rn(x0, c[e]), __fmul_rn(x1, s[e]));
                x1 = __fadd_rn(__fmul_rn(x0, s[e]), __fmul_rn(x1, c[e]));
                x0 = y0;
            }
        }
    }
    const BlockScale b = block_scale(fmaxf(absmax8(x), absmax8(x + 8)), a32);
    uint8_t* codes = const_cast<uint8_t*>(v.codes[t]) + (uint64_t)at * (v.d / 2) + 8 * blk;
    *reinterpret_cast<uint2*>(codes) = make_uint2(encode8(x, b.inv), encode8(x + 8, b.inv));
    const_cast<uint8_t*>(v.scales[t])[(uint64_t)at * (v.d / 16) + blk] = (uint8_t)b.code;
}

__device__ __forceinline__ void gather_block(const RowArgs& a, const RowBlock& r, float a32, uint8_t* dst) {
    const __half2 s2 = e4m3x2_to_half2((uint16_t)(r.x[0].z | (r.x[0].z << 8)));
    uint32_t h[8], o[8];
    decode8(r.x[0].x, s2, h);
    decode8(r.x[0].y, s2, h + 4);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float2 f = __half22float2(bits_h2(h[i]));
        const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(f.x, a32), __fmul_rn(f.y, a32));
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    store32(dst, a.wide, o);
}

template <bool APPEND>
__global__ void __launch_bounds__(kRowWarps * 32, 3) rows_kernel(const __grid_constant__ RowArgs a) {
    constexpr int kInFlight = APPEND ? 4 : 8;
    const View& v = a.v;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int blocks = v.d / 16, per = 32 / blocks;  // lanes of a row, rows of a warp
    const int64_t w = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    const int part = (int)(w % a.parts);
    const int64_t r0 = w / a.parts * per;
    if (r0 >= v.n_rows) return;
    const int last = (int)min((int64_t)v.n_rows, r0 + per) - 1;
    int b = find_seq(v, (int)r0, lane);
    const int b1 = ld_coherent(v.row_start + b + 1) > last ? b : find_seq(v, last, lane);
    const int row = (int)r0 + lane / blocks, blk = lane % blocks;
    if (row > last) return;
    if (b != b1) {  // the rows' own sequences lie between
        int lo = b, hi = b1 + 1;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (ld_coherent(v.row_start + mid) <= row) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    const Seq s = load_seq(v, b);
    if (row < s.first || row - s.first >= s.n) return;  // no sequence's row: left as it was
    const int pos = s.len - s.n + (row - s.first);
    const bool none = pos < 0;  // before the sequence's first position: not written, read as zeros
    if (APPEND && none) return;
    const int page = none ? 0 : page_of(v, b, pos);
    if (page < 0) return;
    // the cache's row of head 0, and a head's distance from the one before it (rows below 2^32: host)
    const int off = none ? 0 : v.page_shift >= 0 ? pos & (v.page_size - 1) : pos % v.page_size;
    const uint32_t at0 = (uint32_t)page * (uint32_t)v.kv_heads * (uint32_t)v.page_size + (uint32_t)off;
    // (read once: behind the stores below the compiler would have to read them again)
    const float a32[2] = {ld_coherent(v.a32[0]), ld_coherent(v.a32[1])};
    const int i0 = (int)((int64_t)a.items * part / a.parts), i1 = (int)((int64_t)a.items * (part + 1) / a.parts);
    for (int i = i0; i < i1; i += kInFlight) {
        RowBlock r[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; u++) {
            const int head = (i + u) >> 1, t = (i + u) & 1;
            if (i + u >= i1) break;
            const uint32_t at = at0 + (uint32_t)head * (uint32_t)v.page_size;
            if (APPEND) {
                const uint8_t* src = a.rows[t] + ((int64_t)row * a.ld[t] + (int64_t)head * v.d + 16 * blk) * 2;
                load32(src, a.wide, r[u].x);
            } else if (none) {
                r[u].x[0] = make_uint4(0u, 0u, 0u, 0u);
            } else {
                const uint2 c = ld_coherent(reinterpret_cast<const uint2*>(v.codes[t] + (uint64_t)at * (v.d / 2) + 8 * blk));
                r[u].x[0] = make_uint4(c.x, c.y, ld_coherent(v.scales[t] + (uint64_t)at * (v.d / 16) + blk), 0u);
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; u++) {
            const int head = (i + u) >> 1, t = (i + u) & 1;
            if (i + u >= i1) break;
            if (APPEND)
                append_block(a, r[u], t, t ? a32[1] : a32[0], row, blk, at0 + (uint32_t)head * (uint32_t)v.page_size);
            else
                gather_block(a, r[u], t ? a32[1] : a32[0],
                             a.rows[t] + ((int64_t)row * a.ld[t] + (int64_t)head * v.d + 16 * blk) * 2);
        }
    }
}

// ---------------------------------------------------------------------------
// attention of few rows.
//
// Unit: one sequence, one K/V head, up to 8 NT rows (row, query head of the
// group); the units' 32-key tiles are dealt out in equal runs, one a warp
// (paged.cuh): warps that wait for nobody hide one another's beginnings and
// ends of units.  Both products have the cache as the A
// operand (S^T = K Q^T, O^T = V^T P^T), so eight rows fill a matrix
// instruction's columns; a lane reads whole 16-byte (K) and 8-byte (V) pieces of
// rows, with the contraction's columns permuted to fit, and P^T comes from S^T
// by an 8 x 8 transpose in registers.  The cache's bytes pass through a ring of
// tiles in shared memory a warp, so that no registers wait for them.
//
// Bound: the cache's bytes (a key and value are 9/8 head_dim bytes a head),
// and beside them the decoding (fp4mma.cuh).  64 sequences of 6000 keys on
// average x 8 heads of 128 (177 MB; calls in a graph): 47 us, of which the runs'
// beginnings and ends (places, pages, queries; joining) are about 11; the copies
// alone then take 27 (6.5 TB/s), the arithmetic alone 31, both 37.
// ---------------------------------------------------------------------------
constexpr int kKeys = 32;  // keys of a tile
constexpr int kSms = 148;
constexpr int kWarps = 4;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Page of the 16 keys from kq on: -1 when no row of the unit sees one of them
// (not looked up), else what the table lists.
__device__ __forceinline__ int group_page(const View& v, const int32_t* table, const Span& sp, int kq) {
    if (!group_seen(sp, kq)) return -1;
    return listed(table, v.page_shift >= 0 ? kq >> v.page_shift : kq / v.page_size);
}

// A warp's ring of 32-key tiles in shared memory, filled by asynchronous
// copies: the tile's K codes, V codes, K scales, V scales.  D = 128: the two
// halves of a V row change places in every other pair of keys, which spreads
// the reads below over all banks.
template <int D>
struct Ring {
    static constexpr int kCodes = kKeys * D / 2, kScales = kKeys * D / 16;
    static constexpr int k = 0, v = kCodes, ks = 2 * kCodes, vs = 2 * kCodes + kScales;
    static constexpr int bytes = 2 * (kCodes + kScales);
};

// 16 bytes to shared memory, those behind the first `n` as zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// A lane's share of a tile's copies: where it reads (add row * (D / 2) or row *
// (D / 16)) and the key that its first chunk belongs to.
template <int D>
struct CopyLane {
    static constexpr int kChunks = D / 32;                // of a row of codes
    static constexpr int kRows = 32 / kChunks;            // rows that the warp copies at a time
    static constexpr int kScaleChunks = kKeys * D / 256;  // of a tensor
    const uint8_t *k, *v, *s;
    uint32_t dk, dv, ds;  // the same in a ring slot
    int key, skey;
    bool scales;
    __device__ __forceinline__ CopyLane(const View& a, int lane) {
        const int c = lane % kChunks, t = lane / kScaleChunks, i = lane % kScaleChunks;
        key = lane / kChunks;
        k = a.codes[0] + key * (D / 2) + 16 * c;
        v = a.codes[1] + key * (D / 2) + 16 * c;
        dk = Ring<D>::k + key * (D / 2) + 16 * c;
        dv = Ring<D>::v + key * (D / 2) + 16 * (D == 128 ? c ^ (key & 2) : c);  // (key & 2 is the same 8 or 16 rows on)
        scales = t < 2;
        skey = i * (256 / D);
        s = a.scales[t & 1] + (skey & (kGroup - 1)) * (D / 16);
        ds = (t ? Ring<D>::vs : Ring<D>::ks) + 16 * i;
    }
};

// Tile at key k0 into a ring slot.  Groups that no row sees, and what lies
// behind the last key (it is not a value), become zeros.
template <int D>
__device__ __forceinline__ void load_tile(const View& v, const CopyLane<D>& ln, int b, uint32_t page_rows,
                                          uint32_t head_row, const Span& sp, int k0, const int* pages, uint32_t dst) {
    constexpr int kRows = CopyLane<D>::kRows;
    uint32_t row[2];
    bool ok[2];
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const int kq = k0 + 16 * q;
        ok[q] = (unsigned)pages[q] < (unsigned)v.n_pages;
        if (!ok[q] && pages[q] != -1) record_error(v.err, NVFP4_ERR_DEVICE, (uint32_t)b);
        const int at = v.page_shift >= 0 ? kq & (v.page_size - 1) : kq % v.page_size;
        row[q] = ok[q] ? (uint32_t)pages[q] * page_rows + head_row + (uint32_t)at : 0u;  // below 2^32 (host)
    }
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const uint8_t *k = ln.k + (uint64_t)row[q] * (D / 2), *w = ln.v + (uint64_t)row[q] * (D / 2);
#pragma unroll
        for (int j = 0; j < 16 / kRows; j++) {
            const int n = ok[q] && k0 + 16 * q + j * kRows + ln.key < sp.hi ? 16 : 0;
            copy16(dst + ln.dk + (16 * q + j * kRows) * (D / 2), k + j * kRows * (D / 2), n);
            copy16(dst + ln.dv + (16 * q + j * kRows) * (D / 2), w + j * kRows * (D / 2), n);
        }
    }
    if (ln.scales) {
        const int n = (ln.skey < 16 ? ok[0] : ok[1]) ? min(16, max(0, sp.hi - k0 - ln.skey) * (D / 16)) : 0;
        copy16(dst + ln.ds, ln.s + (uint64_t)(ln.skey < 16 ? row[0] : row[1]) * (D / 16), n);
    }
}

// The same for a tile of 32 keys that all count and lie in one page of the
// cache, from cache row `row` on.
template <int D>
__device__ __forceinline__ void load_whole_tile(const CopyLane<D>& ln, uint32_t row, uint32_t dst) {
    constexpr int kRows = CopyLane<D>::kRows;
    const uint8_t *k = ln.k + (uint64_t)row * (D / 2), *w = ln.v + (uint64_t)row * (D / 2);
#pragma unroll
    for (int j = 0; j < kKeys / kRows; j++) {
        copy16(dst + ln.dk + j * kRows * (D / 2), k + j * kRows * (D / 2), 16);
        copy16(dst + ln.dv + j * kRows * (D / 2), w + j * kRows * (D / 2), 16);
    }
    if (ln.scales) copy16(dst + ln.ds, ln.s + (uint64_t)(row + (ln.skey & kGroup)) * (D / 16), 16);
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t p, uint32_t* w) {
    if (N == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p));
    else if (N == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(p));
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t p) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(p));
    return x;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t p) {
    uint32_t x;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(p));
    return x;
}

// Which of a group's 16 keys is row r < 8 of the S product (row r + 8: 8 more):
// the transpose hands rows 2 t and 2 t + 1 to lane t, whose V rows then are
// keys t, 4 + (t ^ 1), and 8 more, in four different bank quarters each time.
__device__ __forceinline__ int key_of_row(int r) { return (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1; }

// A key's D / 16 scales
template <int D>
__device__ __forceinline__ void clear_scales(uint32_t p) {
    if (D == 128) asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(p), "r"(0u) : "memory");
    else asm volatile("st.shared.u32 [%0], %1;" ::"r"(p), "r"(0u) : "memory");
}

// One key's D / 4 codes and their scales -> D / 8 pairs
template <int D>
__device__ __forceinline__ void decode_k(const uint32_t* c, uint32_t sc, uint32_t* o) {
    const __half2 s = e4m3x2_to_half2((uint16_t)sc);
    const __half2 s0 = __low2half2(s), s1 = __high2half2(s);
#pragma unroll
    for (int w = 0; w < D / 32; w++) decode8(c[w], w < D / 64 ? s0 : s1, o + 4 * w);
}

// One warp, one piece: kStages tiles in its ring at `ring`.  A piece that is not
// the whole unit goes to slot u.slot of part_o and part_ml.
template <int D, int NT, int kStages>
__device__ __forceinline__ void decode_piece(const AttnArgs& a, const Piece& u, uint32_t ring, float* part_o,
                                             float2* part_ml) {
    constexpr int kCols = 8 * NT, kSteps = D / 16, kPer = D / 8;  // kPer: a lane's channels of O
    const View& v = a.v;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Seq& s = u.s;
    const Rows& rows = u.rows;
    const int b = u.b, head = u.head, f0 = u.f0, begin = u.begin, end = u.end;
    const Tiles<kKeys> tiles(rows.span);

    const uint32_t page_rows = (uint32_t)v.kv_heads * (uint32_t)v.page_size;
    const uint32_t head_row = (uint32_t)head * (uint32_t)v.page_size;
    const CopyLane<D> ln(v, lane);
    const int32_t* table = v.pages + (int64_t)b * v.max_pages;

    // queries: column n of tile j is row f0 + 8 j + n; columns past the last row are zeros and nobody reads them
    uint4 raw[NT][D / 32];
#pragma unroll
    for (int j = 0; j < NT; j++) {
        const int f = f0 + 8 * j + g;
        const bool in = 8 * j + g < rows.n;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((int64_t)(s.first + f / a.group) * a.ld_q + (int64_t)(head * a.group + f % a.group) * D + D / 4 * t) * 2);
#pragma unroll
        for (int i = 0; i < D / 32; i++) raw[j][i] = in ? ld_coherent(src + i) : make_uint4(0u, 0u, 0u, 0u);
    }

    // Copies run kStages - 1 tiles ahead.  A tile whose 32 keys are all seen by some row and
    // lie in one page (of 32 or more tokens) takes the short way.
    const Span& sp = rows.span;
    const int jump = tiles.first > tiles.n_sink ? tiles.n_sink * kKeys : -1, after_jump = tiles.first * kKeys;
    auto step = [&](int k0) { return k0 + kKeys == jump ? after_jump : k0 + kKeys; };  // from the sinks' tiles to the others
    auto whole = [&](int k0) {
        return v.page_shift >= 5 && ((k0 >= sp.lo && k0 + kKeys <= sp.hi) || k0 + kKeys <= sp.sink_end);
    };
    // pages are looked up for 32 tiles at a time, a lane a tile
    int listed0 = -1, listed1 = -1;
    auto lookup = [&](int i) {
        listed0 = listed1 = -1;
        if (i + lane < end) {
            const int k = tiles.key0(i + lane);
            listed0 = group_page(v, table, sp, k);
            listed1 = group_page(v, table, sp, k + kGroup);
        }
    };
    auto fetch = [&](int i, int k0, uint32_t dst) {
        const int page0 = __shfl_sync(0xFFFFFFFFu, listed0, i), page1 = __shfl_sync(0xFFFFFFFFu, listed1, i);
        if (whole(k0) && (unsigned)page0 < (unsigned)v.n_pages) {
            load_whole_tile<D>(ln, (uint32_t)page0 * page_rows + head_row + (uint32_t)(k0 & (v.page_size - 1)), dst);
        } else {
            const int pages[2] = {page0, page1};
            load_tile<D>(v, ln, b, page_rows, head_row, sp, k0, pages, dst);
        }
    };
    const uint32_t ring_end = ring + kStages * Ring<D>::bytes;
    int ahead = begin, ahead_k0 = tiles.key0(begin);  // the next tile to fetch, its page already looked up
    uint32_t dst = ring;
    lookup(begin);
    auto advance = [&]() {
        if (ahead < end) {
            fetch(ahead - begin, ahead_k0, dst);
            dst = dst + Ring<D>::bytes == ring_end ? ring : dst + Ring<D>::bytes;
            ahead_k0 = step(ahead_k0);
            if ((++ahead - begin) % 32 == 0) lookup(ahead);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; i++) advance();

    uint32_t qb[NT][D / 8];
    float c_col[NT][2];
#pragma unroll
    for (int j = 0; j < NT; j++) {
        const float down = scale_row<D / 32>(raw[j], qb[j]) * (ld_coherent(v.a32[0]) * a.scale_log2);
#pragma unroll
        for (int e = 0; e < 2; e++) c_col[j][e] = __shfl_sync(0xFFFFFFFFu, down, 8 * t + 4 * e);
    }
    // a tile from k0 on is seen whole by every row when k0 <= all_hi and k0 >= all_lo or <= all_sink
    const int all_hi = s.len - s.n + f0 / a.group - (kKeys - 1);
    const int all_lo = a.window > 0 ? s.len - s.n + (f0 + rows.n - 1) / a.group - a.window + 1 : 0;
    const int all_sink = a.sinks - kKeys;

    // a column's reference m (paged.cuh) as -m, and what an exponent relative to it must exceed for m to move; before
    // its first visible key m is 0 and any exponent does
    constexpr float kLimit = kLazy + kHead;
    float nm[NT][2], limit[NT][2], l[NT][2], o[NT][kSteps][4];
#pragma unroll
    for (int j = 0; j < NT; j++) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
            nm[j][e] = l[j][e] = 0.0f;
            limit[j][e] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kSteps; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[j][i][e] = 0.0f;
    }

    // the lane's places in a ring slot
    const int kr = key_of_row(g);
    const uint32_t l_k = Ring<D>::k + kr * (D / 2) + D / 8 * t, l_ks = Ring<D>::ks + kr * (D / 16) + D / 64 * t;
    const int v0 = t, v1 = 4 + (t ^ 1);  // keys of a group whose V rows the lane decodes, and 8 more
    const uint32_t l_v0 = Ring<D>::v + v0 * (D / 2) + (D == 128 ? 16 * ((g >> 1) ^ (v0 & 2)) + 8 * (g & 1) : 4 * g);
    const uint32_t l_v1 = Ring<D>::v + v1 * (D / 2) + (D == 128 ? 16 * ((g >> 1) ^ (v1 & 2)) + 8 * (g & 1) : 4 * g);
    const uint32_t l_vs = Ring<D>::vs + (D == 128 ? g : g / 2);
    int k0 = tiles.key0(begin);
    uint32_t at = ring;

#pragma unroll 1
    for (int i = begin; i < end; i++, k0 = step(k0), at = at + Ring<D>::bytes == ring_end ? ring : at + Ring<D>::bytes) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();  // the tile is there for every lane, and every lane has left the slot that is filled next
        advance();
        // places that no row sees (outside the window) may hold anything: their weight is 0, and their values' scale has to be
        if (max(k0, sp.sink_end) < min(k0 + kKeys, sp.lo)) {
            if (k0 + lane >= sp.sink_end && k0 + lane < sp.lo) clear_scales<D>(at + Ring<D>::vs + lane * (D / 16));
            __syncwarp();
        }
        // z: the scores' exponents, relative to the reference: 2^z is the weight
        float z[2][NT][4];
#pragma unroll
        for (int q = 0; q < 2; q++) {
            uint32_t ka[D / 8], kb[D / 8], w[D / 32];
            const uint32_t k16 = at + l_k + 16 * q * (D / 2), s16 = at + l_ks + 16 * q * (D / 16);
            lds_words<D / 32>(k16, w);
            decode_k<D>(w, D == 128 ? lds_u16(s16) : lds_u8(s16) * 0x101u, ka);
            lds_words<D / 32>(k16 + 8 * (D / 2), w);
            decode_k<D>(w, D == 128 ? lds_u16(s16 + 8 * (D / 16)) : lds_u8(s16 + 8 * (D / 16)) * 0x101u, kb);
#pragma unroll
            for (int j = 0; j < NT; j++) {
                mma_16816_first(z[q][j], ka[0], kb[0], ka[1], kb[1], qb[j][0], qb[j][1]);
#pragma unroll
                for (int e = 1; e < kSteps; e++)
                    mma_16816(z[q][j], ka[2 * e], kb[2 * e], ka[2 * e + 1], kb[2 * e + 1], qb[j][2 * e], qb[j][2 * e + 1]);
            }
        }
#pragma unroll
        for (int q = 0; q < 2; q++)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) z[q][j][e] = fmaf(z[q][j][e], c_col[j][e & 1], nm[j][e & 1]);
        // every key of the tile seen by every row, or else key by key
        if (!(k0 <= all_hi && (k0 >= all_lo || k0 <= all_sink))) {
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int p = s.len - s.n + (f0 + 8 * j + 2 * t + e) / a.group;
                    const int lo = a.window > 0 ? p - a.window + 1 : 0;
#pragma unroll
                    for (int q = 0; q < 2; q++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int key = k0 + 16 * q + kr + 8 * h;
                            if (!(key <= p && (key >= lo || key < a.sinks))) z[q][j][2 * h + e] = -INFINITY;
                        }
                }
        }
        float top[NT][2];
        bool over = false;
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                top[j][e] = fmaxf(fmaxf(z[0][j][e], z[0][j][e + 2]), fmaxf(z[1][j][e], z[1][j][e + 2]));
                over |= top[j][e] > limit[j][e];
            }
        if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float mx = top[j][e];
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
                    if (mx > limit[j][e]) {
                        mx -= kHead;
                        const float f = limit[j][e] == kLimit ? ex2(-mx) : 0.0f;
                        limit[j][e] = kLimit;
                        nm[j][e] -= mx;
                        l[j][e] *= f;
#pragma unroll
                        for (int q = 0; q < 2; q++) {
                            z[q][j][e] -= mx;
                            z[q][j][e + 2] -= mx;
                        }
#pragma unroll
                        for (int r = 0; r < kSteps; r++) {
                            o[j][r][e] *= f;
                            o[j][r][e + 2] *= f;
                        }
                    }
                }
        }
#pragma unroll
        for (int q = 0; q < 2; q++) {
            uint32_t pb[NT][2];
#pragma unroll
            for (int j = 0; j < NT; j++) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    p[e] = ex2(z[q][j][e]);
                    l[j][e & 1] += p[e];
                }
                // the weights go to the tensor cores in binary16 (2^-11 of each, 2^-32 of the row's largest: paged.cuh),
                // an eighth of what the result's store in bf16 rounds; binary32 would need a second product of the rest
                pb[j][0] = transpose8x8(h2_bits(__floats2half2_rn(p[0], p[1])));
                pb[j][1] = transpose8x8(h2_bits(__floats2half2_rn(p[2], p[3])));
            }
            // V: channels kPer g .. + kPer - 1 of the lane's four keys, two keys a pair
            uint32_t va[kPer], vb[kPer];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                uint32_t w0[D / 64], w1[D / 64];
                const uint32_t key = 16 * q + 8 * h;
                lds_words<D / 64>(at + l_v0 + key * (D / 2), w0);
                lds_words<D / 64>(at + l_v1 + key * (D / 2), w1);
                const __half2 two = e4m3x2_to_half2((uint16_t)(lds_u8(at + l_vs + (key + v0) * (D / 16)) |
                                                               (lds_u8(at + l_vs + (key + v1) * (D / 16)) << 8)));
#pragma unroll
                for (int e = 0; e < D / 64; e++) decode8_rows(w0[e], w1[e], two, (h ? vb : va) + 8 * e);
            }
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int r = 0; r < kSteps; r++)
                    mma_16816(o[j][r], va[2 * r], va[2 * r + 1], vb[2 * r], vb[2 * r + 1], pb[j][0], pb[j][1]);
        }
    }
    __syncwarp();  // every lane has left the ring (its copies are done: none was begun behind the last tile)

    const float back = ld_coherent(v.a32[1]);
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
            float sum = l[j][e];
#pragma unroll
            for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            const int n = 8 * j + 2 * t + e;  // the lane holds channels kPer g .. of this row
            if (n >= rows.n) continue;
            if (u.slot >= 0) {
                const int64_t at = (int64_t)u.slot * kCols + n;
                float4* dst = reinterpret_cast<float4*>(part_o + at * D + kPer * g);
#pragma unroll
                for (int r = 0; r < kSteps; r += 2)
                    dst[r / 2] = make_float4(o[j][r][e], o[j][r][e + 2], o[j][r + 1][e], o[j][r + 1][e + 2]);
                if (g == 0) part_ml[at] = make_float2(limit[j][e] == kLimit ? -nm[j][e] : kFloor, sum);
            } else {
                const float f = sum == 0.0f ? 0.0f : __fdiv_rn(back, sum);  // a row that sees no key: zeros
                const int row = s.first + (f0 + n) / a.group, qh = head * a.group + (f0 + n) % a.group;
                uint4* dst = reinterpret_cast<uint4*>(a.o + ((int64_t)row * a.ld_o + (int64_t)qh * D + kPer * g) * 2);
#pragma unroll
                for (int r = 0; r < kSteps; r += 4) {
                    uint32_t y[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(o[j][r + i][e] * f, o[j][r + i][e + 2] * f);
                        y[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    dst[r / 4] = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
}

// CTAs of a launch: three an SM (two with 16 columns) by registers and shared memory.
template <int NT>
constexpr int decode_ctas() {
    return kSms * (NT == 1 ? 3 : 2);
}
constexpr int kDecodeStages = 4;
constexpr int kLeast = 3;  // tiles of a run: fewer make many pieces to join, more few warps (one sequence of 6000 keys, 8
                           // heads of 128: 17.4 us with 3, 18.1 with 4, 21 with 8; of 16000: 26 with 2, 22.8 with 3)
template <int D>
constexpr int decode_smem() {
    return kWarps * kDecodeStages * Ring<D>::bytes;
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 3 : 2) decode_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(128) uint8_t ring_mem[];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    RunScratch<kWarps * 32>& scratch = *reinterpret_cast<RunScratch<kWarps * 32>*>(ring_mem);
    const int warp = threadIdx.x >> 5;
    const uint32_t ring = smem_u32(ring_mem) + (uint32_t)(warp * kDecodeStages * Ring<D>::bytes);
    Run run = make_run<8 * NT, kKeys, kWarps * 32, kWarps>(a, warp, kLeast, scratch);
    __syncthreads();  // the rings take the scratch memory over
    Piece u;
    int4 cut = make_int4(0, 0, 0, 0);
    while (next_piece<8 * NT, kKeys>(a, run, u)) {
        decode_piece<D, NT, kDecodeStages>(a, u, ring, a.part_o, a.part_ml);
        if (u.pieces) cut = make_int4(u.pieces, u.pair, u.head, u.rows.n);
    }
    if ((threadIdx.x & 31) == 0) a.cut[run.worker] = cut;
}

// Short sequences: a unit a CTA, its tiles shared out among eight warps that
// join in shared memory, so that one launch does.  Up to 64 tiles (2048 keys)
// it is the faster way (1, 8 and 64 sequences of 8 heads of 128: 700 keys 7.4,
// 8.8, 18.9 us against 15.3, 18.9, 22.8 with runs; 1500 keys 11.1, 14.9, 32
// against 14.6, 18.6, 35; 3000 keys 18.0, 26.1, 54.1 against 16.0, 17.9, 54.4),
// and sequences much shorter than the longest cost it little.  Longer ones take it
// too where a window makes their spans alike and the units fill one wave of CTAs
// to three quarters or more (windows of 4096 of 8 heads, 128 and 64 wide: 32
// sequences 39 and 25 us against 45 and 30 with runs; 24: 38.5 and 24.8 against
// 36.1 and 25.5; 48, which need two waves: 58 and 40 against 57 and 41).
constexpr int kUnitWarps = 8, kUnitStages = 2;
constexpr int kUnitTiles = 64;  // the longest sequence (tiles) that takes this way
template <int D>
constexpr int unit_smem() {
    // (a warp leaves its piece, up to 16 columns, where its ring was)
    static_assert(16 * (D * 4 + 8) <= kUnitStages * Ring<D>::bytes, "piece");
    return kUnitWarps * kUnitStages * Ring<D>::bytes;
}

template <int D, int NT>
__global__ void __launch_bounds__(kUnitWarps * 32, NT == 1 ? 2 : 1) unit_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int kCols = 8 * NT, kBytes = kUnitStages * Ring<D>::bytes;
    extern __shared__ __align__(128) uint8_t ring_mem[];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const View& v = a.v;
    const int warp = threadIdx.x >> 5;
    Piece u;
    int real = 0;
    const int pair = (int)(blockIdx.x / (unsigned)v.kv_heads);
    u.head = (int)(blockIdx.x % (unsigned)v.kv_heads);
    if (pair_tiles<kCols, kKeys>(a, pair, &u.s, &u.rows, &real) == 0) return;
    u.b = pair / a.row_tiles;
    u.f0 = pair % a.row_tiles * kCols;
    u.begin = real * warp / kUnitWarps;
    u.end = real * (warp + 1) / kUnitWarps;
    u.slot = 0;
    float* part = reinterpret_cast<float*>(ring_mem + warp * kBytes);
    decode_piece<D, NT, kUnitStages>(a, u, smem_u32(ring_mem) + (uint32_t)(warp * kBytes), part,
                                     reinterpret_cast<float2*>(part + kCols * D));
    __syncthreads();
    const float back = ld_coherent(v.a32[1]);
    for (int i = threadIdx.x; i < u.rows.n * (D / 2); i += kUnitWarps * 32) {
        const int n = i / (D / 2), d = i % (D / 2) * 2;
        float mx = kFloor, sum = 0.0f, y0 = 0.0f, y1 = 0.0f;
#pragma unroll
        for (int w = 0; w < kUnitWarps; w++)
            mx = fmaxf(mx, reinterpret_cast<const float2*>(ring_mem + w * kBytes + kCols * D * 4)[n].x);
#pragma unroll
        for (int w = 0; w < kUnitWarps; w++) {
            const float2 ml = reinterpret_cast<const float2*>(ring_mem + w * kBytes + kCols * D * 4)[n];
            const float2 x = *reinterpret_cast<const float2*>(ring_mem + w * kBytes + (n * D + d) * 4);
            const float f = ex2(ml.x - mx);
            sum += ml.y * f;
            y0 += x.x * f;
            y1 += x.y * f;
        }
        const int row = u.s.first + (u.f0 + n) / a.group, qh = u.head * a.group + (u.f0 + n) % a.group;
        const float f = sum == 0.0f ? 0.0f : __fdiv_rn(back, sum);  // a row that sees no key: zeros
        *reinterpret_cast<__nv_bfloat162*>(a.o + ((int64_t)row * a.ld_o + (int64_t)qh * D + d) * 2) =
            __floats2bfloat162_rn(y0 * f, y1 * f);
    }
}

// Joins the pieces of the unit that worker blockIdx.x began, a warp a row.  It is
// loads that wait for loads (place, then weights and pieces together), so as many
// as registers hold are on the way: one piece after the other it took 7 and 14 us
// behind the decode steps of 64 and 4 sequences, 5 and 8 so.
template <int D, int COLS>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnArgs a) {
    const View& v = a.v;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kBatch = COLS == kChunkRows ? 2 : 8;  // (a unit of chunks rarely lies in more than two runs)
    const int4 cut = __ldcg(a.cut + blockIdx.x);
    const int lane = threadIdx.x & 31, n = (int)blockIdx.y * 8 + (threadIdx.x >> 5);
    // (a record or row range that something else has overwritten meanwhile must not lead outside the tensors)
    if (cut.x <= 0 || cut.x > (int)(gridDim.x - blockIdx.x) || n >= min(cut.w, COLS)) return;
    const int b = cut.y / a.row_tiles;
    if ((unsigned)b >= (unsigned)v.n_seqs || (unsigned)cut.z >= (unsigned)v.kv_heads) return;
    const int first = ld_coherent(v.row_start + b);
    // piece 0 is the end of this worker's run, piece p the beginning of the p-th later one's
    auto at = [&](int p) { return (int64_t)(2 * ((int)blockIdx.x + p) + (p == 0)) * COLS + n; };
    float mx = kFloor, sum = 0.0f, y[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; e++) y[e] = 0.0f;
    for (int p0 = 0; p0 < cut.x; p0 += 32) {
        // a lane has the weight of one piece; kBatch pieces are on the way at a time
        const int count = min(32, cut.x - p0);
        const float2 ml = lane < count ? __ldcg(a.part_ml + at(p0 + lane)) : make_float2(kFloor, 0.0f);
        float2 x[kBatch][D / 64];
        auto load = [&](int p) {
#pragma unroll
            for (int u = 0; u < kBatch; u++)
#pragma unroll
                for (int e = 0; e < D / 64; e++)
                    x[u][e] = p + u < count ? __ldcg(reinterpret_cast<const float2*>(a.part_o + at(p0 + p + u) * D) + 32 * e + lane)
                                            : make_float2(0.0f, 0.0f);
        };
        load(0);
        float top = fmaxf(mx, ml.x);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const float before = ex2(mx - top), w = lane < count ? ex2(ml.x - top) : 0.0f;
        mx = top;
        float add = ml.y * w;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) add += __shfl_xor_sync(0xFFFFFFFFu, add, d);
        sum = sum * before + add;
#pragma unroll
        for (int e = 0; e < D / 32; e++) y[e] *= before;
        for (int p = 0; p < count; p += kBatch) {
            if (p > 0) load(p);
#pragma unroll
            for (int u = 0; u < kBatch; u++) {
                const float wp = __shfl_sync(0xFFFFFFFFu, w, p + u);
#pragma unroll
                for (int e = 0; e < D / 64; e++) {
                    y[2 * e] += x[u][e].x * wp;
                    y[2 * e + 1] += x[u][e].y * wp;
                }
            }
        }
    }
    const float f2 = sum == 0.0f ? 0.0f : __fdiv_rn(ld_coherent(v.a32[1]), sum);
    const int f = cut.y % a.row_tiles * COLS + n;
    const int64_t row = (int64_t)first + f / a.group, qh = (int64_t)cut.z * a.group + f % a.group;
    if (row < 0 || row >= v.n_rows) return;
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(a.o + (row * a.ld_o + qh * D) * 2);
#pragma unroll
    for (int e = 0; e < D / 64; e++) dst[32 * e + lane] = __floats2bfloat162_rn(y[2 * e] * f2, y[2 * e + 1] * f2);
}

}  // namespace paged
}  // namespace nvfp4

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
using namespace nvfp4;
using namespace nvfp4::paged;

namespace {

constexpr size_t kControl = 256;

bool odd(const void* p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// Programmatic dependent launch: the grid's start overlaps the previous
// kernel's end; every kernel here waits for it before it reads or writes.
template <class Args>
nvfp4_status launch_dependent(void (*kernel)(Args), dim3 grid, int threads, int smem, cudaStream_t stream, const Args& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return NVFP4_ERR_CUDA;
    }
    return NVFP4_OK;
}

// The checks of the cache and the rows that all three calls share.
nvfp4_status check_paged(const nvfp4_paged_cache* c, const nvfp4_paged_rows* r, const void* ws, size_t ws_bytes,
                         size_t need) {
    if (!c || !r || !ws || ws_bytes < need) return NVFP4_ERR_INVALID_ARG;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !c->k_global || !c->v_global || c->n_pages <= 0 ||
        c->page_size <= 0 || c->kv_heads <= 0)
        return NVFP4_ERR_INVALID_ARG;
    if (r->n_seqs < 0 || r->n_rows < 0 || r->max_pages < 0 || r->max_rows < 0 || r->max_len < 0)
        return NVFP4_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return NVFP4_ERR_UNSUPPORTED;
    if (c->page_size % kGroup != 0 || c->page_size > (1 << 20) || c->kv_heads > (1 << 16) || r->n_rows > (1 << 30) ||
        r->max_len > (1 << 30) || (int64_t)c->n_pages * c->kv_heads > (((int64_t)1 << 32) - 1) / c->page_size)
        return NVFP4_ERR_UNSUPPORTED;
    if (r->n_seqs > 0 && r->n_rows > 0 && (!r->row_start || !r->lens || (r->max_pages > 0 && !r->pages)))
        return NVFP4_ERR_INVALID_ARG;
    if (odd(c->k_codes, 15u) || odd(c->k_scales, 15u) || odd(c->v_codes, 15u) || odd(c->v_scales, 15u) ||
        odd(c->k_global, 3u) || odd(c->v_global, 3u) || odd(r->row_start, 3u) || odd(r->lens, 3u) || odd(r->pages, 3u) ||
        odd(ws, 255u))
        return NVFP4_ERR_MISALIGNED;
    return NVFP4_OK;
}

View make_view(const nvfp4_paged_cache* c, const nvfp4_paged_rows* r, void* record) {
    View v{};
    v.codes[0] = static_cast<const uint8_t*>(c->k_codes);
    v.codes[1] = static_cast<const uint8_t*>(c->v_codes);
    v.scales[0] = static_cast<const uint8_t*>(c->k_scales);
    v.scales[1] = static_cast<const uint8_t*>(c->v_scales);
    v.a32[0] = c->k_global;
    v.a32[1] = c->v_global;
    v.row_start = r->row_start;
    v.lens = r->lens;
    v.pages = r->pages;
    v.n_pages = c->n_pages;
    v.page_size = c->page_size;
    v.page_shift = -1;
    for (int i = 0; i < 31; i++)
        if (c->page_size == 1 << i) v.page_shift = i;
    v.kv_heads = c->kv_heads;
    v.d = c->head_dim;
    v.n_seqs = r->n_seqs;
    v.max_pages = r->max_pages;
    v.n_rows = r->n_rows;
    v.room = (int)std::min<int64_t>((int64_t)r->max_pages * c->page_size, 1 << 30);
    v.err = static_cast<DevError*>(record);
    return v;
}

nvfp4_status rows_call(bool append, const nvfp4_paged_cache* c, const nvfp4_paged_rows* r, const void* k, int64_t ld_k,
                       const void* v, int64_t ld_v, const float* rope_cos, const float* rope_sin, void* ws,
                       size_t ws_bytes, nvfp4_stream_t stream) {
    const nvfp4_status st = check_paged(c, r, ws, ws_bytes, kControl);
    if (st != NVFP4_OK) return st;
    const int64_t width = (int64_t)c->kv_heads * c->head_dim;
    if (ld_k < width || ld_v < width || (rope_cos == nullptr) != (rope_sin == nullptr)) return NVFP4_ERR_INVALID_ARG;
    if (r->n_rows == 0 || r->n_seqs == 0) return NVFP4_OK;
    if (!k || !v) return NVFP4_ERR_INVALID_ARG;
    if (odd(k, 15u) || odd(v, 15u) || ld_k % 8 != 0 || ld_v % 8 != 0 || odd(rope_cos, 15u) || odd(rope_sin, 15u))
        return NVFP4_ERR_MISALIGNED;
    RowArgs a{};
    a.v = make_view(c, r, ws);
    a.rows[0] = static_cast<uint8_t*>(const_cast<void*>(k));
    a.rows[1] = static_cast<uint8_t*>(const_cast<void*>(v));
    a.ld[0] = ld_k;
    a.ld[1] = ld_v;
    a.rope_cos = rope_cos;
    a.rope_sin = rope_sin;
    a.wide = !odd(k, 31u) && !odd(v, 31u) && ld_k % 16 == 0 && ld_v % 16 == 0;
    const int64_t per = 512 / c->head_dim, groups = (r->n_rows + per - 1) / per;  // rows of a warp
    // one wave of 24 warps an SM (what append's registers allow), then more heads a warp
    a.items = 2 * c->kv_heads;
    a.parts = (int)std::min<int64_t>(a.items, std::max<int64_t>(1, (int64_t)kSms * 24 / groups));
    const int64_t grid = (groups * a.parts + kRowWarps - 1) / kRowWarps;
    if (grid >= ((int64_t)1 << 31)) return NVFP4_ERR_UNSUPPORTED;
    return launch_dependent(append ? rows_kernel<true> : rows_kernel<false>, dim3((unsigned)grid), kRowWarps * 32, 0,
                            (cudaStream_t)stream, a);
}

// How an attention call is launched; the same for its workspace query.
struct Plan {
    bool chunks;  // chunk_kernel (paged_attention.cu), else decode_kernel
    bool units;   // unit_kernel: no pieces
    int cols;     // (row, query head) pairs of a unit
    int row_tiles, ctas, workers;
    size_t cut, ml, o, ws;  // bytes from the workspace's start
};

bool make_plan(const nvfp4_paged_cache* c, const nvfp4_paged_rows* r, int heads, int window, int sinks, Plan* p) {
    const int64_t pairs = (int64_t)r->max_rows * (heads / c->kv_heads);
    if (pairs >= ((int64_t)1 << 31)) return false;
    // More pairs than the decode kernel's 16 columns would read (and decode) the keys several times
    p->chunks = pairs > 16;
    p->cols = p->chunks ? kChunkRows : pairs <= 8 ? 8 : 16;
    p->row_tiles = (int)std::max<int64_t>(1, (pairs + p->cols - 1) / p->cols);
    if ((int64_t)p->row_tiles * std::max(1, r->n_seqs) >= ((int64_t)1 << 31) - 1024) return false;
    p->ctas = p->chunks ? kChunkCtas : p->cols == 8 ? decode_ctas<1>() : decode_ctas<2>();
    // no more CTAs than the shortest runs of the most tiles
    int64_t seen = r->max_len;
    if (window > 0) seen = std::min<int64_t>(seen, (int64_t)window + sinks + std::min<int64_t>(r->max_rows, p->cols));
    const int keys = p->chunks ? kChunkKeys : kKeys, least = p->chunks ? kChunkLeast : kWarps * kLeast;
    p->workers = p->chunks ? 1 : kWarps;  // of a CTA
    const int64_t tiles = (seen / keys + 3) * p->row_tiles * std::max(1, r->n_seqs);  // ragged at both ends and the sinks'
    p->ctas = (int)std::min<int64_t>(p->ctas, (tiles * c->kv_heads + least - 1) / least);
    const int64_t units = (int64_t)p->row_tiles * std::max(1, r->n_seqs) * c->kv_heads;
    const int64_t wave = kSms * (p->cols == 8 ? 2 : 1);
    const bool alike = seen < r->max_len && units <= wave && 4 * units >= 3 * wave;
    p->units = !p->chunks && (seen / keys < kUnitTiles || alike) && units < ((int64_t)1 << 31);
    if (p->units) {
        p->ctas = (int)units;
        p->workers = 0;
    }
    p->cut = kControl;
    p->workers *= p->units ? 0 : p->ctas;
    p->ml = p->cut + (size_t)p->workers * sizeof(int4);
    p->o = p->ml + (size_t)p->workers * 2 * p->cols * sizeof(float2);
    p->ws = p->o + (size_t)p->workers * 2 * p->cols * c->head_dim * sizeof(float);
    return true;
}

nvfp4_status check_heads(const nvfp4_paged_cache* c, int heads, int window, int sinks) {
    if (heads <= 0 || heads % c->kv_heads != 0 || window < 0 || sinks < 0) return NVFP4_ERR_INVALID_ARG;
    if (heads > (1 << 16) || window > (1 << 30) || sinks > (1 << 30)) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

}  // namespace

extern "C" nvfp4_status nvfp4_paged_append(const nvfp4_paged_cache* cache, const nvfp4_paged_rows* rows,
                                           const void* k_bf16, int64_t ld_k, const void* v_bf16, int64_t ld_v,
                                           const float* rope_cos, const float* rope_sin, void* workspace,
                                           size_t ws_bytes, nvfp4_stream_t stream) {
    return rows_call(true, cache, rows, k_bf16, ld_k, v_bf16, ld_v, rope_cos, rope_sin, workspace, ws_bytes, stream);
}

extern "C" nvfp4_status nvfp4_paged_gather(const nvfp4_paged_cache* cache, const nvfp4_paged_rows* rows, void* k_bf16,
                                           int64_t ld_k, void* v_bf16, int64_t ld_v, void* workspace, size_t ws_bytes,
                                           nvfp4_stream_t stream) {
    return rows_call(false, cache, rows, k_bf16, ld_k, v_bf16, ld_v, nullptr, nullptr, workspace, ws_bytes, stream);
}

extern "C" size_t nvfp4_paged_attention_workspace_bytes(const nvfp4_paged_cache* cache, const nvfp4_paged_rows* rows,
                                                        int32_t heads, int32_t window, int32_t sinks) {
    Plan p;
    if (!cache || !rows || cache->kv_heads <= 0 || (cache->head_dim != 64 && cache->head_dim != 128) ||
        rows->n_seqs < 0 || rows->n_rows < 0 || rows->max_rows < 0 || rows->max_len < 0 ||
        check_heads(cache, heads, window, sinks) != NVFP4_OK || !make_plan(cache, rows, heads, window, sinks, &p))
        return 0;
    return p.ws;
}

extern "C" nvfp4_status nvfp4_paged_attention(const nvfp4_paged_cache* cache, const nvfp4_paged_rows* rows,
                                              const void* q_bf16, int64_t ld_q, int32_t heads, int32_t window,
                                              int32_t sinks, float scale, void* o_bf16, int64_t ld_o, void* workspace,
                                              size_t ws_bytes, nvfp4_stream_t stream) {
    return nvfp4_paged_attention_recorded(cache, rows, q_bf16, ld_q, heads, window, sinks, scale, o_bf16, ld_o, workspace,
                                          ws_bytes, workspace, stream);
}

extern "C" nvfp4_status nvfp4_paged_attention_recorded(const nvfp4_paged_cache* cache, const nvfp4_paged_rows* rows,
                                                       const void* q_bf16, int64_t ld_q, int32_t heads, int32_t window,
                                                       int32_t sinks, float scale, void* o_bf16, int64_t ld_o,
                                                       void* workspace, size_t ws_bytes, void* record,
                                                       nvfp4_stream_t stream) {
    nvfp4_status st = check_paged(cache, rows, workspace, ws_bytes, kControl);
    if (st != NVFP4_OK) return st;
    st = check_heads(cache, heads, window, sinks);
    if (st != NVFP4_OK) return st;
    if (!record) return NVFP4_ERR_INVALID_ARG;
    if (odd(record, 255u)) return NVFP4_ERR_MISALIGNED;
    const int64_t width = (int64_t)heads * cache->head_dim;
    if (!(scale >= 0.0f) || std::isinf(scale) || ld_q < width || ld_o < width) return NVFP4_ERR_INVALID_ARG;
    Plan p;
    if (!make_plan(cache, rows, heads, window, sinks, &p)) return NVFP4_ERR_UNSUPPORTED;
    if (ws_bytes < p.ws) return NVFP4_ERR_INVALID_ARG;
    if (rows->n_rows == 0 || rows->n_seqs == 0 || rows->max_rows == 0) return NVFP4_OK;
    if (!q_bf16 || !o_bf16) return NVFP4_ERR_INVALID_ARG;
    if (odd(q_bf16, 15u) || odd(o_bf16, 15u) || ld_q % 8 != 0 || ld_o % 8 != 0) return NVFP4_ERR_MISALIGNED;
    AttnArgs a{};
    a.v = make_view(cache, rows, record);
    a.q = static_cast<const uint8_t*>(q_bf16);
    a.o = static_cast<uint8_t*>(o_bf16);
    a.ld_q = ld_q;
    a.ld_o = ld_o;
    a.group = heads / cache->kv_heads;
    a.window = window;
    a.sinks = window > 0 ? sinks : 0;
    a.max_rows = rows->max_rows;
    a.row_tiles = p.row_tiles;
    const float sc = scale > 0.0f ? scale : 1.0f / sqrtf((float)cache->head_dim);
    a.scale_log2 = sc * 1.4426950408889634f;  // log2(e)
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.cut = reinterpret_cast<int4*>(ws + p.cut);
    a.part_ml = reinterpret_cast<float2*>(ws + p.ml);
    a.part_o = reinterpret_cast<float*>(ws + p.o);
    if (p.chunks) {
        st = launch_chunks(a, (unsigned)p.ctas, (cudaStream_t)stream);
        if (st != NVFP4_OK) return st;
    } else {
        static PerDevice<int> ready;
        int done = 0;
        st = ready.get(&done, [](int, int& v) {
            v = 1;
            auto room = [](void (*f)(AttnArgs), int bytes) {
                return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
            };
            return room(decode_kernel<128, 1>, decode_smem<128>()) && room(decode_kernel<128, 2>, decode_smem<128>()) &&
                           room(decode_kernel<64, 1>, decode_smem<64>()) && room(decode_kernel<64, 2>, decode_smem<64>()) &&
                           room(unit_kernel<128, 1>, unit_smem<128>()) && room(unit_kernel<128, 2>, unit_smem<128>()) &&
                           room(unit_kernel<64, 1>, unit_smem<64>()) && room(unit_kernel<64, 2>, unit_smem<64>())
                       ? NVFP4_OK
                       : NVFP4_ERR_CUDA;
        });
        if (st != NVFP4_OK) return st;
        const bool wide = cache->head_dim == 128, one = p.cols == 8;
        if (p.units)
            return launch_dependent(wide ? (one ? unit_kernel<128, 1> : unit_kernel<128, 2>)
                                         : (one ? unit_kernel<64, 1> : unit_kernel<64, 2>),
                                    dim3((unsigned)p.ctas), kUnitWarps * 32, wide ? unit_smem<128>() : unit_smem<64>(),
                                    (cudaStream_t)stream, a);
        st = launch_dependent(wide ? (one ? decode_kernel<128, 1> : decode_kernel<128, 2>)
                                   : (one ? decode_kernel<64, 1> : decode_kernel<64, 2>),
                              dim3((unsigned)p.ctas), kWarps * 32, wide ? decode_smem<128>() : decode_smem<64>(),
                              (cudaStream_t)stream, a);
        if (st != NVFP4_OK) return st;
    }
    void (*join)(AttnArgs) =
        cache->head_dim == 128
            ? (p.chunks ? combine_kernel<128, kChunkRows> : p.cols == 8 ? combine_kernel<128, 8> : combine_kernel<128, 16>)
            : (p.chunks ? combine_kernel<64, kChunkRows> : p.cols == 8 ? combine_kernel<64, 8> : combine_kernel<64, 16>);
    return launch_dependent(join, dim3((unsigned)p.workers, (unsigned)(p.cols / 8)), 256, 0, (cudaStream_t)stream, a);
}
