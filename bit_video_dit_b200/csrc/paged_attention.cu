// Causal attention of chunks of new tokens over the paged NVFP4 cache on the
// tensor cores (few rows a head: paged.cu).
//
// Work unit: one sequence, one K/V head and two tiles (A and B) of 128 (row,
// query head of the group) pairs, so that a group's heads share the keys; the
// units' 64-key tiles are dealt out in equal runs (paged.cuh), one a CTA and
// SM.  Inside a CTA
//   warps 0-3   softmax of tile A (thread = pair = TMEM lane),
//   warps 4-7   softmax of tile B,
//   warps 8-15  producers: a thread decodes a quarter of one key's row of K and
//               of V a tile straight into the operands' layout,
//   warps 16-17 a thread each issuing A's and B's tcgen05 products and commits.
// The decoding costs as many instructions as the softmax's arithmetic, and one
// warp a scheduler cannot issue it fast enough, hence eight producer warps.
// Registers: 640 threads start with 96 each; the producers give 32 of theirs to
// the softmax (setmaxnreg).
// Shared memory: Q_A, Q_B, K[2], V[4], P_A[2], P_B[2], each of 8 x 8 core
// matrices without swizzle, element (row r, column c) at (c / 8) * rows * 16 + r
// * 16 + (c % 8) * 2: Q, K and P K-major, V MN-major.  TMEM: S_A[2], S_B[2] (64
// columns each) and O_A, O_B.  Scores are double-buffered: QK(j + 2) is issued
// as soon as the softmax has read S of tile j, so that it finds the next tile's
// done.  One buffer of 128 keys and one issuing thread took 4% more, rows read and
// written a lane a row another 2%.  2640 rows x 24 heads over 23760 visible keys:
// 723 us in a graph that repeats one input (950 TFLOP/s of what the rows see), 730
// with inputs in turn, 762 back to back from Python with inputs in turn.
// What is left is no unit's rate (products 1280 cycles of a tile's 2300,
// exponentials 1024, issue 45%) but the hand-overs between the roles: without
// the softmax's and the producers' work the same barriers take 0.93 of the time.
// Measured and not taken (times against the kernel then): 16 softmax warps (each
// half a tile's columns; 1.48), four issuing threads (1.09), a lane waiting for its
// warp (1.18), an eighth of the exponentials as polynomials (1.08).
// The softmax takes one pass a tile against a reference 7 binary orders below the
// largest score (paged.cuh) that moves only when a row's weights in the tile sum
// above 2^15 (binary16 holds those below).  Every wait is bounded; a timeout
// records NVFP4_ERR_TIMEOUT and every role stops.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fp4mma.cuh"
#include "paged.cuh"

namespace nvfp4 {
namespace paged {

using namespace fp4mma;

namespace {

constexpr int kTile = 128;          // pairs of a query tile
constexpr int kKeys = kChunkKeys;   // keys of a key tile
constexpr int kKBufs = 2, kVBufs = 4;
constexpr int kAhead = 2;  // tiles whose bytes are on the way in a producer's registers
constexpr int kProducer0 = 8, kMmaWarp = 16;  // first producer warp, the issuing warps
constexpr int kThreads = 640;                 // five warpgroups
constexpr int kProducers = 256, kSoft = 128;  // producer threads, threads of a softmax group
constexpr int kLaunchRegs = 96, kSoftRegs = 128, kProducerRegs = 64;  // the last warpgroup keeps kLaunchRegs
static_assert(2 * kSoftRegs + 2 * kProducerRegs + kLaunchRegs <= 5 * kLaunchRegs, "registers of the block");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0, kOCol = 256;
constexpr float kPMax = 32768.0f;  // a tile's weights summing above 2^15 make the row check its maximum
constexpr uint64_t kLimitNs = 2000000000ull;

template <int D>
struct Smem {
    static constexpr int kQ = kTile * D * 2, kKV = kKeys * D * 2, kP = kTile * kKeys * 2;
    static constexpr uint32_t q = 0, k = 2 * kQ, v = k + kKBufs * kKV, p = v + kVBufs * kKV;
    static constexpr int bytes = p + 4 * kP;
};

// kind::f16, binary32 accumulator, binary16 operands, A K-major, B K-major (0)
// or MN-major (1), M = 128
__host__ __device__ constexpr uint32_t idesc(int b_mn, int n) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

// The words of a shared-memory matrix descriptor (common.cuh, smem_desc, no
// swizzle): the low one holds the address, so that a product of an unrolled run
// costs one addition an operand.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14); }

// D[tmem] = A B (ACC: D += A B), 16 of the contraction's columns.
template <bool ACC>
__device__ __forceinline__ void mma_step(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                         uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t"
        "}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}

struct Shared {
    uint64_t q_full[2];       // softmax X -> MMA: Q_X of the unit written (128 arrivals)
    uint64_t s_full[2][2];    // MMA -> softmax X: S_X[i] done (commit), and so is every product issued before it
    uint64_t p_full[2][2];    // softmax X -> MMA: P_X[i] written, S_X[i] read, O_X rescaled (128)
    uint64_t pv_done[2][2];   // MMA -> softmax X: the product of P_X[i] into O_X done (commit)
    uint64_t k_full[kKBufs];  // producers -> MMA: K buffer written (256)
    uint64_t k_empty[kKBufs]; // MMA -> producers: A's and B's product of the K buffer done (2 arrivals)
    uint64_t v_full[kVBufs];  // producers -> MMA: V buffer written (256)
    uint64_t v_empty[kVBufs]; // MMA -> producers: A's and B's product of the V buffer done (2)
    uint64_t done[2];         // every product issued for A, for B is done (before TMEM is freed)
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, Shared& sh, const AttnArgs& a,
                                             uint32_t where) {
    volatile int* abort = &sh.abort;
    if (mbar_wait_bounded(bar, parity, abort, kLimitNs)) return true;
    record_error(a.v.err, NVFP4_ERR_TIMEOUT, where);
    *abort = 1;
    return false;
}

// ---- producers -------------------------------------------------------------
// A quarter of one key's row of K or V as stored.
template <int D>
struct Part {
    uint32_t c[D / 32];  // D / 4 codes
    uint32_t sc;         // their scales (D = 128: two bytes, 64: one)
};

template <int D>
struct PartKV {
    Part<D> k, v;
};

// What the page table lists for key `row` of tile i (looked at only when its
// bytes are fetched), -1 when no row of the unit sees it.
__device__ __forceinline__ int lookup(const View& v, const int32_t* table, const Piece& w, const Tiles<kKeys>& tiles, int i,
                                      int row) {
    const int key = tiles.key0(i) + row;
    const Span& s = w.rows.span;
    if (i >= w.end || key >= s.hi || (key < s.lo && key >= s.sink_end)) return -1;
    return listed(table, v.page_shift >= 0 ? key >> v.page_shift : key / v.page_size);
}

template <int D>
__device__ __forceinline__ void fetch(const View& v, const Piece& w, const Tiles<kKeys>& tiles, int i, int row, int page,
                                      int part, PartKV<D>& x) {
    if ((unsigned)page < (unsigned)v.n_pages) {
        const int key = tiles.key0(i) + row;
        const int at = v.page_shift >= 0 ? key & (v.page_size - 1) : key % v.page_size;
        const uint32_t r =
            ((uint32_t)page * (uint32_t)v.kv_heads + (uint32_t)w.head) * (uint32_t)v.page_size + (uint32_t)at;
#pragma unroll
        for (int t = 0; t < 2; t++) {
            Part<D>& h = t ? x.v : x.k;
            const uint8_t* pc = v.codes[t] + (uint64_t)r * (D / 2) + part * (D / 8);
            const uint8_t* ps = v.scales[t] + (uint64_t)r * (D / 16) + part * (D / 64);
            if (D == 128) {
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(pc));
                h.c[0] = q.x, h.c[1] = q.y, h.c[2] = q.z, h.c[3] = q.w;
                h.sc = __ldg(reinterpret_cast<const uint16_t*>(ps));
            } else {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(pc));
                h.c[0] = q.x, h.c[1] = q.y;
                h.sc = __ldg(ps);
            }
        }
    } else {
        if (page != -1) record_error(v.err, NVFP4_ERR_DEVICE, (uint32_t)w.b);
#pragma unroll
        for (int e = 0; e < D / 32; e++) x.k.c[e] = x.v.c[e] = 0u;
        x.k.sc = x.v.sc = 0u;
    }
}

// Its values e2m1 s (exact in binary16) into the operand at `base`.
template <int D>
__device__ __forceinline__ void store_part(const Part<D>& h, uint32_t base, int row, int part) {
    const __half2 two = e4m3x2_to_half2((uint16_t)h.sc);
#pragma unroll
    for (int w = 0; w < D / 32; w++) {  // 8 channels each
        uint32_t o[4];
        decode8(h.c[w], w >= 2 ? __high2half2(two) : __low2half2(two), o);
        st_shared16(base + (part * (D / 32) + w) * (kKeys * 16) + row * 16, make_uint4(o[0], o[1], o[2], o[3]));
    }
}

template <int D>
__device__ __forceinline__ void producer_role(const AttnArgs& a, Shared& sh, uint32_t smem0, int tid, Run run) {
    const int row = tid & (kKeys - 1), part = tid / kKeys;
    uint32_t n = 0u;  // tiles so far
    Piece w;
    while (next_piece<kChunkRows, kKeys>(a, run, w)) {
        if (w.begin >= w.end) continue;
        const Tiles<kKeys> tiles(w.rows.span);
        // data is loaded kAhead tiles ahead, its place looked up kAhead tiles before that
        PartKV<D> x[kAhead];
        int page[kAhead];
        const int32_t* table = a.v.pages + (int64_t)w.b * a.v.max_pages;
#pragma unroll
        for (int u = 0; u < kAhead; u++) page[u] = lookup(a.v, table, w, tiles, w.begin + u, row);
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            fetch<D>(a.v, w, tiles, w.begin + u, row, page[u], part, x[u]);
            page[u] = lookup(a.v, table, w, tiles, w.begin + u + kAhead, row);
        }
        for (int i0 = w.begin; i0 < w.end; i0 += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; u++) {
                const int i = i0 + u;
                if (i >= w.end) break;
                const uint32_t kb = n % kKBufs, vb = n % kVBufs;
                // a buffer's first fill passes at once (parity 1 of a fresh barrier)
                if (!wait_or_stop(&sh.k_empty[kb], ((n / kKBufs) & 1u) ^ 1u, sh, a, 4)) return;
                store_part<D>(x[u].k, smem0 + Smem<D>::k + kb * Smem<D>::kKV, row, part);
                fence_proxy_async_smem();
                mbar_arrive(&sh.k_full[kb]);
                if (!wait_or_stop(&sh.v_empty[vb], ((n / kVBufs) & 1u) ^ 1u, sh, a, 5)) return;
                store_part<D>(x[u].v, smem0 + Smem<D>::v + vb * Smem<D>::kKV, row, part);
                fence_proxy_async_smem();
                mbar_arrive(&sh.v_full[vb]);
                n++;
                fetch<D>(a.v, w, tiles, i + kAhead, row, page[u], part, x[u]);
                page[u] = lookup(a.v, table, w, tiles, i + 2 * kAhead, row);
            }
        }
    }
}

// ---- softmax ---------------------------------------------------------------
// The warp's 32 pairs from f on into Q at rows row0 .. (zeros past the last),
// scaled by 2^k to binary16 (fp4mma.cuh); returns 2^-k of the lane's row.  Four
// lanes read 64 bytes of a row together: a lane a row, the loads of 32 lines an
// instruction took 2 us a unit, the stores of O below 4.
template <int D>
__device__ __forceinline__ float load_q_rows(const AttnArgs& a, const Piece& w, uint32_t q_s, int f, int row0) {
    constexpr int kParts = D / 32;  // of 64 bytes
    const int lane = threadIdx.x & 31, c = lane & 3;
    uint4 v[4][kParts];
    float down[4];
#pragma unroll
    for (int g = 0; g < 4; g++) {
        const int fr = f + 8 * g + (lane >> 2);
        const bool in = fr < w.f0 + w.rows.n;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((int64_t)(w.s.first + fr / a.group) * a.ld_q + (int64_t)(w.head * a.group + fr % a.group) * D) * 2) + c;
#pragma unroll
        for (int i = 0; i < kParts; i++) v[g][i] = in ? __ldg(src + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int g = 0; g < 4; g++) {
        uint32_t mx = max_bits<kParts>(v[g]);
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const RowScale rs = row_scale(mx);
        down[g] = rs.down;
#pragma unroll
        for (int i = 0; i < kParts; i++) {
            uint32_t x[4];
            scale8(v[g][i], rs.up, x);
            st_shared16(q_s + (4 * i + c) * 2048 + (row0 + 8 * g + (lane >> 2)) * 16, make_uint4(x[0], x[1], x[2], x[3]));
        }
    }
    float mine = 0.0f;
#pragma unroll
    for (int g = 0; g < 4; g++) {
        const float x = __shfl_sync(0xFFFFFFFFu, down[g], 4 * (lane & 7));
        if (lane >> 3 == g) mine = x;
    }
    return mine;
}

// 128 bytes of each lane's row, by way of 4 KB of shared memory at `at`, to the
// rows' places `dst` (NULL: none), so that eight lanes write a row's line.
__device__ __forceinline__ void store_rows(uint32_t at, const uint32_t* x, uint8_t* dst) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; i++)
        st_shared16(at + lane * 128 + ((i ^ (lane & 7)) << 4), make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
    __syncwarp();
    const int c = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = 4 * i + (lane >> 3);
        uint4 y;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                     : "r"(at + r * 128 + ((c ^ (r & 7)) << 4)));
        uint8_t* p = reinterpret_cast<uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(dst), r));
        if (p) *reinterpret_cast<uint4*>(p + 16 * c) = y;
    }
    __syncwarp();
}

// What a row sees of a tile: keys below `hi` that are at least `lo` or below
// `sink` (all relative to the tile).
struct RowMask {
    int lo, hi, sink;
    // bits of the 32 keys from 32 c on
    __device__ __forceinline__ uint32_t bits(int c) const {
        auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; };
        return below(hi - 32 * c) & (~below(lo - 32 * c) | below(sink - 32 * c));
    }
};

template <bool MASK>
__device__ __forceinline__ float tile_max(uint32_t t_s, const RowMask& rm) {
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < kKeys / 32; c++) {
        uint32_t r[32];
        tmem_ld_32cols(t_s + 32 * c, r);
        const uint32_t seen = MASK ? rm.bits(c) : 0xFFFFFFFFu;
        tmem_ld_wait();
        tmem_regs_ready(r);
#pragma unroll
        for (int j = 0; j < 32; j++)
            if (!MASK || (seen >> j) & 1u) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(r[j]));
    }
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// P row: 2^(c_s s - m), zero where the row does not see the key, in binary16
// at row `row`; returns the sum of the unrounded values.
template <bool MASK>
__device__ __forceinline__ float write_p(uint32_t t_s, uint32_t p_s, int row, const RowMask& rm, float c_s, float m) {
    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    const float2 cc = make_float2(c_s, c_s), mm = make_float2(-m, -m);
    uint32_t rc[kKeys / 32][32];
#pragma unroll
    for (int c = 0; c < kKeys / 32; c++) tmem_ld_32cols(t_s + 32 * c, rc[c]);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < kKeys / 32; c++) {
        tmem_regs_ready(rc[c]);
        const uint32_t seen = MASK ? rm.bits(c) : 0xFFFFFFFFu;
#pragma unroll
        for (int q4 = 0; q4 < 4; q4++) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int j = 8 * q4 + 2 * e;
                const float2 t = fma2(make_float2(__uint_as_float(rc[c][j]), __uint_as_float(rc[c][j + 1])), cc, mm);
                float2 p = make_float2(ex2(t.x), ex2(t.y));
                if (MASK) {
                    if (!((seen >> j) & 1u)) p.x = 0.0f;
                    if (!((seen >> (j + 1)) & 1u)) p.y = 0.0f;
                }
                sum[e & 1] = add2(sum[e & 1], p);
                w[e] = h2_bits(__floats2half2_rn(p.x, p.y));
            }
            st_shared16(p_s + (4 * c + q4) * 2048 + row * 16, make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
    return (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
}

template <int D>
__device__ __forceinline__ void softmax_role(const AttnArgs& a, Shared& sh, uint32_t smem0, uint32_t tmem, int X, int row,
                                             Run run) {
    const uint32_t lane_off = (uint32_t)(row & ~31) << 16;
    const uint32_t t_s0 = tmem + kSCol + 2 * kKeys * X + lane_off, t_o = tmem + kOCol + 128 * X + lane_off;
    const uint32_t q_s = smem0 + Smem<D>::q + X * Smem<D>::kQ, p_s0 = smem0 + Smem<D>::p + 2 * X * Smem<D>::kP;
    const float ck = __ldg(a.v.a32[0]) * a.scale_log2, back = __ldg(a.v.a32[1]);
    uint32_t n = 0u;  // tiles so far
    Piece w;
    while (next_piece<kChunkRows, kKeys>(a, run, w)) {
        if (X == 1 && w.rows.n <= kTile) continue;  // no tile B
        const Tiles<kKeys> tiles(w.rows.span);
        const int f = w.f0 + X * kTile + row;
        const bool real = f < w.f0 + w.rows.n;
        float c_s = 0.0f;
        if (w.begin < w.end) {  // (without a key tile the issuing thread does not wait for it)
            c_s = load_q_rows<D>(a, w, q_s, f - (row & 31), row & ~31) * ck;
            fence_proxy_async_smem();
            mbar_arrive(&sh.q_full[X]);
        }
        const int p = w.s.len - w.s.n + f / a.group;
        const int hi = real ? p + 1 : 0, lo = a.window > 0 ? p - a.window + 1 : 0;
        // a tile from k0 on is seen whole by the warp's rows when hi_min >= k0 + 64 and (lo_max <= k0 or in the sinks);
        // padding rows compute as if they saw everything
        const int hi_min = __reduce_min_sync(0xFFFFFFFFu, real ? hi : 0x7FFFFFFF);
        const int lo_max = __reduce_max_sync(0xFFFFFFFFu, real ? lo : 0);
        float m = -INFINITY, l = 0.0f;
        bool first = true;
        for (int i = w.begin; i < w.end; i++, n++) {
            const int k0 = tiles.key0(i);
            const uint32_t buf = n & 1u, ph = (n >> 1) & 1u;
            const uint32_t t_s = t_s0 + kKeys * buf, p_s = p_s0 + buf * Smem<D>::kP;
            const RowMask rm{lo - k0, hi - k0, a.sinks - k0};
            const bool all = hi_min >= k0 + kKeys && (lo_max <= k0 || a.sinks >= k0 + kKeys);
            // (a wait's outcome is made uniform over the warp: the TMEM loads are warp-collective)
            const bool got = __all_sync(0xFFFFFFFFu, wait_or_stop(&sh.s_full[X][buf], ph, sh, a, 1));
            if (!got) return;
            tc_fence_after();
            float tsum = all ? write_p<false>(t_s, p_s, row, rm, c_s, m) : write_p<true>(t_s, p_s, row, rm, c_s, m);
            const bool redo = !(tsum <= kPMax);
            if (__any_sync(0xFFFFFFFFu, redo)) {
                // tcgen05.ld / st are warp-collective: the whole warp takes part
                const float mt = (all ? tile_max<false>(t_s, rm) : tile_max<true>(t_s, rm)) * c_s;  // c_s >= 0
                float factor = 1.0f;
                // (a sum above 2^15 means a score more than 9 above m; m 7 below the largest brings it to 2^13 at most)
                if (redo && mt - m > kLazy) {
                    factor = ex2(m - (mt - kHead));  // 0 on the first tile (m = -inf)
                    l *= factor;
                    m = mt - kHead;
                }
                if (!first && __any_sync(0xFFFFFFFFu, factor != 1.0f)) {
                    // the last tile's product may still be adding to O
                    if (!__all_sync(0xFFFFFFFFu, wait_or_stop(&sh.pv_done[X][buf ^ 1u], ((n - 1) >> 1) & 1u, sh, a, 3))) return;
                    tc_fence_after();
                    uint32_t o[32];
#pragma unroll 1
                    for (int c = 0; c < D / 32; c++) {
                        tmem_ld_32cols(t_o + 32 * c, o);
                        tmem_ld_wait();
                        tmem_regs_ready(o);
#pragma unroll
                        for (int j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * factor);
                        tmem_st_32cols(t_o + 32 * c, o);
                    }
                    tmem_st_wait();
                }
                tsum = all ? write_p<false>(t_s, p_s, row, rm, c_s, m) : write_p<true>(t_s, p_s, row, rm, c_s, m);
            }
            l += tsum;
            // S read, O rescaled and P written before the MMA thread goes on
            tc_fence_before();
            fence_proxy_async_smem();
            mbar_arrive(&sh.p_full[X][buf]);
            first = false;
        }
        if (!first) {
            const bool got = __all_sync(0xFFFFFFFFu, wait_or_stop(&sh.pv_done[X][(n - 1) & 1u], ((n - 1) >> 1) & 1u, sh, a, 2));
            if (!got) return;
            tc_fence_after();
        }
        const float inv_l = l == 0.0f ? 0.0f : __fdiv_rn(back, l);  // a row that sees no key: zeros
        const int64_t slot = (int64_t)w.slot * kChunkRows + f - w.f0;
        uint8_t* dst = nullptr;
        if (real && w.slot >= 0) {
            a.part_ml[slot] = make_float2(m, l);
            dst = reinterpret_cast<uint8_t*>(a.part_o + slot * D);
        } else if (real) {
            dst = a.o + ((int64_t)(w.s.first + f / a.group) * a.ld_o + (int64_t)(w.head * a.group + f % a.group) * D) * 2;
        }
        // through P: no product reads it now, and the next unit's first P is written when all four warps have signalled
        // q_full behind this
        const uint32_t stage = p_s0 + (row >> 5) * 4096;
        auto load_o = [&](int c, uint32_t* r) {
            if (!first) {
                tmem_ld_32cols(t_o + 32 * c, r);
                tmem_ld_wait();
                tmem_regs_ready(r);
            } else {
#pragma unroll
                for (int j = 0; j < 32; j++) r[j] = 0u;
            }
        };
        if (w.slot >= 0) {
#pragma unroll 1
            for (int c = 0; c < D / 32; c++) {
                uint32_t r[32];
                load_o(c, r);
                store_rows(stage, r, dst ? dst + 128 * c : nullptr);
            }
        } else {
#pragma unroll 1
            for (int c = 0; c < D / 64; c++) {
                uint32_t x[32];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    uint32_t r[32];
                    load_o(2 * c + h, r);
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[2 * j]) * inv_l,
                                                                       __uint_as_float(r[2 * j + 1]) * inv_l);
                        x[16 * h + j] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                }
                store_rows(stage, x, dst ? dst + 128 * c : nullptr);
            }
        }
        // O read before the next unit's first product overwrites it
        tc_fence_before();
    }
}

// ---- the issuing thread ----------------------------------------------------
// One thread issues tile A's products, another tile B's.  A thread that waits
// on a barrier after a commit leaves the tensor cores some 100 cycles without
// work (measured: 391 cycles for a batch of four that takes 256); the other's
// products fill them.  Per unit: QK(0) and QK(1), then per key tile j: PV(j),
// QK(j+2).  The hazards:
//  - QK(j+2) overwrites S_X[j & 1]: issued only after p_full[X][j & 1] of tile j
//    (its softmax has read it);
//  - softmax X(j) writes P_X[j & 1] once s_full[X][j & 1] has fired, which covers
//    PV(j-2), issued by the same thread before QK(j);
//  - it rescales O_X only after pv_done[X] of tile j - 1 (PV(j) comes after p_full);
//  - K and V buffers are released (k_empty, v_empty) by both threads, by the
//    commit of their product or, in a unit without a tile B, at once;
//  - a unit's first products overwrite S_X, Q_X and O_X: q_full[X] of the unit
//    is signalled after softmax X has read the last unit's O_X.
template <int D>
__device__ __forceinline__ void mma_role(const AttnArgs& a, Shared& sh, uint32_t smem0, uint32_t tmem, int X, Run run) {
    constexpr uint32_t ID_QK = idesc(0, kKeys), ID_PV = idesc(1, D);
    // n: the CTA's tile (K and V buffers), x: the tile of A or B (S and P buffers)
    const uint32_t q_lo = desc_lo(smem0 + Smem<D>::q + X * Smem<D>::kQ, 2048), k_lo = desc_lo(smem0 + Smem<D>::k, kKeys * 16);
    const uint32_t p_lo = desc_lo(smem0 + Smem<D>::p + 2 * X * Smem<D>::kP, 2048), v_lo = desc_lo(smem0 + Smem<D>::v, 128);
    const uint32_t o = tmem + kOCol + 128 * X, s0 = tmem + kSCol + 2 * kKeys * X;
    auto qk = [&](uint32_t n, uint32_t x) {
        const uint32_t kx = k_lo + n % kKBufs * (Smem<D>::kKV >> 4), s = s0 + kKeys * (x & 1u);
        mma_step<false>(s, q_lo, desc_hi(128), kx, desc_hi(128), ID_QK);
#pragma unroll
        for (int k = 1; k < D / 16; k++)
            mma_step<true>(s, q_lo + k * (4096 >> 4), desc_hi(128), kx + k * (2 * kKeys * 16 >> 4), desc_hi(128), ID_QK);
        tc_commit(&sh.s_full[X][x & 1u]);
        tc_commit(&sh.k_empty[n % kKBufs]);
    };
    auto pv = [&](uint32_t n, uint32_t x, bool acc) {
        const uint32_t px = p_lo + (x & 1u) * (Smem<D>::kP >> 4), vx = v_lo + n % kVBufs * (Smem<D>::kKV >> 4);
        if (acc) mma_step<true>(o, px, desc_hi(128), vx, desc_hi(kKeys * 16), ID_PV);
        else mma_step<false>(o, px, desc_hi(128), vx, desc_hi(kKeys * 16), ID_PV);
#pragma unroll
        for (int k = 1; k < kKeys / 16; k++)
            mma_step<true>(o, px + k * (4096 >> 4), desc_hi(128), vx + k * (256 >> 4), desc_hi(kKeys * 16), ID_PV);
        tc_commit(&sh.pv_done[X][x & 1u]);
        tc_commit(&sh.v_empty[n % kVBufs]);
    };
    auto k_ready = [&](uint32_t n) { return wait_or_stop(&sh.k_full[n % kKBufs], (n / kKBufs) & 1u, sh, a, 7); };
    auto v_ready = [&](uint32_t n) { return wait_or_stop(&sh.v_full[n % kVBufs], (n / kVBufs) & 1u, sh, a, 8); };
    int4 cut = make_int4(0, 0, 0, 0);
    uint32_t ph_q = 0u, n = 0u, x = 0u;  // tiles so far, and those of A or B
    bool ok = true;
    Piece w;
    while (ok && next_piece<kChunkRows, kKeys>(a, run, w)) {
        if (w.pieces) cut = make_int4(w.pieces, w.pair, w.head, w.rows.n);
        const int count = max(0, w.end - w.begin);
        if (count == 0) continue;
        if (X == 1 && w.rows.n <= kTile) {  // no tile B: only the buffers' release
            for (int j = 0; j < count && ok; j++, n++) {
                ok = k_ready(n);
                if (ok) mbar_arrive(&sh.k_empty[n % kKBufs]);
                ok = ok && v_ready(n);
                if (ok) mbar_arrive(&sh.v_empty[n % kVBufs]);
            }
            continue;
        }
        ok = wait_or_stop(&sh.q_full[X], ph_q, sh, a, 6);
        ph_q ^= 1u;
        for (int j = 0; j < 2 && j < count && ok; j++) {
            ok = k_ready(n + j);
            if (!ok) break;
            tc_fence_after();
            qk(n + j, x + j);
        }
        for (int j = 0; j < count && ok; j++, n++, x++) {
            ok = v_ready(n) && wait_or_stop(&sh.p_full[X][x & 1u], (x >> 1) & 1u, sh, a, 9);
            if (!ok) break;
            tc_fence_after();
            pv(n, x, j > 0);
            if (j + 2 < count) {
                ok = k_ready(n + 2);
                if (!ok) break;
                tc_fence_after();
                qk(n + 2, x + 2);
            }
        }
    }
    if (X == 0) a.cut[blockIdx.x] = cut;
    // every product issued is done before the TMEM is released (also after a stop)
    tc_commit(&sh.done[X]);
    volatile int never = 0;
    if (!mbar_wait_bounded(&sh.done[X], 0, &never, kLimitNs)) record_error(a.v.err, NVFP4_ERR_TIMEOUT, 10);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Shared sh;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    RunScratch<kThreads>& scratch = *reinterpret_cast<RunScratch<kThreads>*>(smem);  // before the operands are there
    const int warp = threadIdx.x >> 5;
    const Run run = make_run<kChunkRows, kKeys, kThreads, 1>(a, 0, kChunkLeast, scratch);
    if (threadIdx.x == 0) {
        for (int X = 0; X < 2; X++) {
            mbar_init(&sh.q_full[X], kSoft);
            mbar_init(&sh.done[X], 1);
            for (int i = 0; i < 2; i++) {
                mbar_init(&sh.pv_done[X][i], 1);
                mbar_init(&sh.s_full[X][i], 1);
                mbar_init(&sh.p_full[X][i], kSoft);
            }
        }
        for (int i = 0; i < kKBufs; i++) {
            mbar_init(&sh.k_full[i], kProducers);
            mbar_init(&sh.k_empty[i], 2);
        }
        for (int i = 0; i < kVBufs; i++) {
            mbar_init(&sh.v_full[i], kProducers);
            mbar_init(&sh.v_empty[i], 2);
        }
        sh.abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base, smem0 = smem_u32(smem);
    if (warp < kProducer0) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        softmax_role<D>(a, sh, smem0, tmem, warp >> 2, threadIdx.x & (kSoft - 1), run);
    } else if (warp < kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        producer_role<D>(a, sh, smem0, threadIdx.x - kProducer0 * 32, run);
    } else if (warp < kMmaWarp + 2 && (threadIdx.x & 31) == 0) {
        mma_role<D>(a, sh, smem0, tmem, warp - kMmaWarp, run);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
nvfp4_status launch(const AttnArgs& a, unsigned ctas, cudaStream_t stream) {
    static PerDevice<int> ready;
    int done = 0;
    const nvfp4_status st = ready.get(&done, [](int, int& v) {
        cudaFuncAttributes at;
        v = 1;
        if (cudaFuncSetAttribute(chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes) !=
                cudaSuccess ||
            cudaFuncGetAttributes(&at, chunk_kernel<D>) != cudaSuccess)
            return NVFP4_ERR_CUDA;
        // the warpgroups' shares are cut from what the block is launched with
        return at.numRegs == kLaunchRegs ? NVFP4_OK : NVFP4_ERR_UNSUPPORTED;
    });
    if (st != NVFP4_OK) return st;
    // (no programmatic launch: the kernel ahead has ended, so the read-only loads above are sound)
    chunk_kernel<D><<<ctas, kThreads, Smem<D>::bytes, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace

nvfp4_status launch_chunks(const AttnArgs& a, unsigned ctas, cudaStream_t stream) {
    return a.v.d == 128 ? launch<128>(a, ctas, stream) : launch<64>(a, ctas, stream);
}

}  // namespace paged
}  // namespace nvfp4
