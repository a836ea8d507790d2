// Causal attention of chunks of new tokens over the paged NVFP4 cache on the
// tensor cores (few rows a head: paged.cu).
//
// Work unit: one sequence, one K/V head and two tiles (A and B) of 128 (row,
// query head of the group) pairs, so that a group's heads share the keys; the
// units' 128-key tiles are dealt out in equal runs (paged.cuh), one a CTA and
// SM.  Inside a CTA
//   warps 0-3   softmax of tile A (thread = pair = TMEM lane),
//   warps 4-7   softmax of tile B,
//   warps 8-15  producers: a thread decodes half of one key's row of K and of V
//               a tile straight into the operands' layout,
//   warp 16     one thread issuing the tcgen05 products and their commits.
// The decoding is what the tensor cores wait for most: a unit pays 2 * 128 * d
// elements of it for 4 * 256 * 128 * d operations, and one warp a scheduler
// cannot issue it fast enough, hence eight producer warps.
// Registers: 640 threads start with 96 each; the producers give 16 of theirs to
// the softmax (setmaxnreg).
// Shared memory: Q_A, Q_B, K, V[2], P_A, P_B, each of 8 x 8 core matrices
// without swizzle, element (row r, column c) at (c / 8) * 2048 + r * 16 +
// (c % 8) * 2: Q, K and P K-major, V MN-major.  TMEM: S_A, S_B and O_A, O_B,
// 128 columns each.  Products in the order PV_A(j), QK_A(j+1), PV_B(j),
// QK_B(j+1): while one tile's softmax runs the tensor cores have the other's.
// The softmax takes one pass a tile against a reference maximum that moves
// only when a row's weights in the tile sum above 2^15 (binary16 holds those
// below).  Every wait is bounded; a timeout records NVFP4_ERR_TIMEOUT and every
// role stops.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fp4mma.cuh"
#include "paged.cuh"

namespace nvfp4 {
namespace paged {

using namespace fp4mma;

namespace {

constexpr int kTile = 128;  // pairs of a query tile, keys of a key tile
constexpr int kProducer0 = 8, kMmaWarp = 16;  // first producer warp, the issuing warp
constexpr int kThreads = 640;                 // five warpgroups
constexpr int kProducers = 256, kSoft = 128;  // producer threads, threads of a softmax group
constexpr int kLaunchRegs = 96, kSoftRegs = 112, kProducerRegs = 80;  // the last warpgroup keeps kLaunchRegs
static_assert(2 * kSoftRegs + 2 * kProducerRegs + kLaunchRegs <= 5 * kLaunchRegs, "registers of the block");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 0, kOCol = 256;
constexpr float kPMax = 32768.0f;  // a tile's weights summing above 2^15 make the row check its maximum
constexpr uint64_t kLimitNs = 2000000000ull;

template <int D>
struct Smem {
    static constexpr int kOperand = kTile * D * 2;  // Q, K, V tiles
    static constexpr int kP = kTile * kTile * 2;
    static constexpr uint32_t q = 0, k = 2 * kOperand, v = 3 * kOperand, p = 5 * kOperand;
    static constexpr int bytes = 5 * kOperand + 2 * kP;
};

// kind::f16, binary32 accumulator, binary16 operands, A K-major, B K-major (0)
// or MN-major (1), M = 128
__host__ __device__ constexpr uint32_t idesc(int b_mn, int n) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

struct Shared {
    uint64_t q_full[2];   // softmax X -> MMA: Q_X of the unit written (128 arrivals)
    uint64_t s_full[2];   // MMA -> softmax X: S_X done (commit), so is every earlier product
    uint64_t p_full[2];   // softmax X -> MMA: P_X written, S_X read, O_X rescaled (128)
    uint64_t o_full[2];   // MMA -> softmax X: the unit's last product into O_X done (commit)
    uint64_t k_full;      // producers -> MMA: K tile written (256)
    uint64_t k_empty;     // MMA -> producers: both products of the K tile done (commit)
    uint64_t v_full[2];   // producers -> MMA: V buffer written (256)
    uint64_t v_empty[2];  // MMA -> producers: both products of the V buffer done (commit)
    uint64_t done;        // every product issued is done (before TMEM is freed)
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
// Half of one key's row of K or V as stored.
template <int D>
struct HalfRow {
    uint4 c[D / 64];
    uint32_t sc;  // D / 32 scale bytes
};

template <int D>
struct HalfKV {
    HalfRow<D> k, v;
};

template <int D>
__device__ __forceinline__ void fetch(const AttnArgs& a, const Piece& w, const Tiles<kTile>& tiles, int i, int row, int half, HalfKV<D>& x) {
    const View& v = a.v;
    const int key = tiles.key0(i) + row;
    int page = -1;
    if (key < w.rows.span.hi && group_seen(w.rows.span, key & ~(kGroup - 1))) page = page_of(v, w.b, key);
    if (page >= 0) {
        const int64_t r = cache_row(v, page, w.head, key);
#pragma unroll
        for (int t = 0; t < 2; t++) {
            HalfRow<D>& h = t ? x.v : x.k;
            const uint4* pc = reinterpret_cast<const uint4*>(v.codes[t] + r * (D / 2) + half * (D / 4));
#pragma unroll
            for (int e = 0; e < D / 64; e++) h.c[e] = __ldg(pc + e);
            const uint8_t* ps = v.scales[t] + r * (D / 16) + half * (D / 32);
            h.sc = D == 128 ? __ldg(reinterpret_cast<const uint32_t*>(ps)) : __ldg(reinterpret_cast<const uint16_t*>(ps));
        }
    } else {
#pragma unroll
        for (int e = 0; e < D / 64; e++) x.k.c[e] = x.v.c[e] = make_uint4(0u, 0u, 0u, 0u);
        x.k.sc = x.v.sc = 0u;
    }
}

// Its values e2m1 s (exact in binary16) into the operand at `base`.
template <int D>
__device__ __forceinline__ void store_half(const HalfRow<D>& h, uint32_t base, int row, int half) {
#pragma unroll
    for (int w = 0; w < D / 16; w++) {  // 8 channels each
        const uint4& q = h.c[w / 4];
        const uint32_t c = (w & 3) == 0 ? q.x : (w & 3) == 1 ? q.y : (w & 3) == 2 ? q.z : q.w;
        const __half2 two = e4m3x2_to_half2((uint16_t)(h.sc >> (16 * (w / 4))));
        uint32_t o[4];
        decode8(c, ((w / 2) & 1) ? __high2half2(two) : __low2half2(two), o);
        st_shared16(base + (half * (D / 16) + w) * 2048 + row * 16, make_uint4(o[0], o[1], o[2], o[3]));
    }
}

template <int D>
__device__ __forceinline__ void producer_role(const AttnArgs& a, Shared& sh, uint32_t smem0, int tid, Run run) {
    const int row = tid & (kTile - 1), half = tid / kTile;
    uint32_t ph_k = 0u, nv = 0u;
    Piece w;
    while (next_piece<kChunkRows, kTile>(a, run, w)) {
        if (w.begin >= w.end) continue;
        const Tiles<kTile> tiles(w.rows.span);
        HalfKV<D> x;
        fetch<D>(a, w, tiles, w.begin, row, half, x);
        for (int i = w.begin; i < w.end; i++) {
            HalfKV<D> next;
            if (i + 1 < w.end) fetch<D>(a, w, tiles, i + 1, row, half, next);
            // a buffer's first fill passes at once (parity 1 of a fresh barrier)
            if (!wait_or_stop(&sh.k_empty, ph_k ^ 1u, sh, a, 4)) return;
            ph_k ^= 1u;
            store_half<D>(x.k, smem0 + Smem<D>::k, row, half);
            fence_proxy_async_smem();
            mbar_arrive(&sh.k_full);
            const uint32_t vb = nv & 1u;
            if (!wait_or_stop(&sh.v_empty[vb], ((nv >> 1) & 1u) ^ 1u, sh, a, 5)) return;
            store_half<D>(x.v, smem0 + Smem<D>::v + vb * Smem<D>::kOperand, row, half);
            fence_proxy_async_smem();
            mbar_arrive(&sh.v_full[vb]);
            nv++;
            x = next;
        }
    }
}

// ---- softmax ---------------------------------------------------------------
// Pair f of the unit's sequence into Q at row `row` (zeros past the last),
// scaled by 2^k to binary16 (fp4mma.cuh); returns 2^-k.
template <int D>
__device__ __forceinline__ float load_q_row(const AttnArgs& a, const Piece& w, uint32_t q_s, int f, int row) {
    uint4 v[D / 8];
    if (f < w.f0 + w.rows.n) {
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + ((int64_t)(w.s.first + f / a.group) * a.ld_q + (int64_t)(w.head * a.group + f % a.group) * D) * 2);
#pragma unroll
        for (int c = 0; c < D / 8; c++) v[c] = __ldg(src + c);
    } else {
#pragma unroll
        for (int c = 0; c < D / 8; c++) v[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    const RowScale rs = row_scale(max_bits<D / 8>(v));
#pragma unroll
    for (int c = 0; c < D / 8; c++) {
        uint32_t x[4];
        scale8(v[c], rs.up, x);
        st_shared16(q_s + c * 2048 + row * 16, make_uint4(x[0], x[1], x[2], x[3]));
    }
    return rs.down;
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
    for (int c = 0; c < 4; c++) {
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
#pragma unroll 1
    for (int c = 0; c < 4; c++) {
        uint32_t rc[32];
        tmem_ld_32cols(t_s + 32 * c, rc);
        const uint32_t seen = MASK ? rm.bits(c) : 0xFFFFFFFFu;
        tmem_ld_wait();
        tmem_regs_ready(rc);
#pragma unroll
        for (int q4 = 0; q4 < 4; q4++) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int j = 8 * q4 + 2 * e;
                const float2 t = fma2(make_float2(__uint_as_float(rc[j]), __uint_as_float(rc[j + 1])), cc, mm);
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
    const uint32_t t_s = tmem + kSCol + 128 * X + lane_off, t_o = tmem + kOCol + 128 * X + lane_off;
    const uint32_t q_s = smem0 + Smem<D>::q + X * Smem<D>::kOperand, p_s = smem0 + Smem<D>::p + X * Smem<D>::kP;
    const float ck = __ldg(a.v.a32[0]) * a.scale_log2, back = __ldg(a.v.a32[1]);
    uint32_t ph_s = 0u, ph_o = 0u;
    Piece w;
    while (next_piece<kChunkRows, kTile>(a, run, w)) {
        if (X == 1 && w.rows.n <= kTile) continue;  // no tile B
        const Tiles<kTile> tiles(w.rows.span);
        const int f = w.f0 + X * kTile + row;
        const bool real = f < w.f0 + w.rows.n;
        float c_s = 0.0f;
        if (w.begin < w.end) {  // (without a key tile the issuing thread does not wait for it)
            c_s = load_q_row<D>(a, w, q_s, f, row) * ck;
            fence_proxy_async_smem();
            mbar_arrive(&sh.q_full[X]);
        }
        const int p = w.s.len - w.s.n + f / a.group;
        const int hi = real ? p + 1 : 0, lo = a.window > 0 ? p - a.window + 1 : 0;
        float m = -INFINITY, l = 0.0f;
        bool first = true;
        for (int i = w.begin; i < w.end; i++) {
            const int k0 = tiles.key0(i);
            const RowMask rm{lo - k0, hi - k0, a.sinks - k0};
            // (padding rows compute as if they saw everything)
            const bool all = __all_sync(0xFFFFFFFFu, !real || (rm.hi >= kTile && (rm.lo <= 0 || rm.sink >= kTile)));
            // (a wait's outcome is made uniform over the warp: the TMEM loads are warp-collective)
            const bool got = __all_sync(0xFFFFFFFFu, wait_or_stop(&sh.s_full[X], ph_s, sh, a, 1));
            ph_s ^= 1u;
            if (!got) return;
            tc_fence_after();
            float tsum = all ? write_p<false>(t_s, p_s, row, rm, c_s, m) : write_p<true>(t_s, p_s, row, rm, c_s, m);
            const bool redo = !(tsum <= kPMax);
            if (__any_sync(0xFFFFFFFFu, redo)) {
                // tcgen05.ld / st are warp-collective: the whole warp takes part
                const float mt = (all ? tile_max<false>(t_s, rm) : tile_max<true>(t_s, rm)) * c_s;  // c_s >= 0
                float factor = 1.0f;
                if (redo && mt - m > kLazy) {
                    factor = ex2(m - mt);  // 0 on the first tile (m = -inf)
                    l *= factor;
                    m = mt;
                }
                if (!first && __any_sync(0xFFFFFFFFu, factor != 1.0f)) {
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
            mbar_arrive(&sh.p_full[X]);
            first = false;
        }
        if (!first) {
            const bool got = __all_sync(0xFFFFFFFFu, wait_or_stop(&sh.o_full[X], ph_o, sh, a, 2));
            ph_o ^= 1u;
            if (!got) return;
            tc_fence_after();
        }
        const int64_t orow = w.s.first + f / a.group;
        const int qh = w.head * a.group + f % a.group;
        const int64_t slot = (int64_t)w.slot * kChunkRows + f - w.f0;
        const float inv_l = l > 0.0f ? __fdiv_rn(back, l) : 0.0f;  // a row that sees no key: zeros
        if (w.slot >= 0 && real) a.part_ml[slot] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < D / 32; c++) {
            uint32_t r[32];
            if (!first) {
                tmem_ld_32cols(t_o + 32 * c, r);
                tmem_ld_wait();
                tmem_regs_ready(r);
            } else {
#pragma unroll
                for (int j = 0; j < 32; j++) r[j] = 0u;
            }
            if (!real) continue;
            if (w.slot >= 0) {
                float4* dst = reinterpret_cast<float4*>(a.part_o + slot * D + 32 * c);
#pragma unroll
                for (int g = 0; g < 8; g++)
                    dst[g] = make_float4(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1]),
                                         __uint_as_float(r[4 * g + 2]), __uint_as_float(r[4 * g + 3]));
            } else {
                uint4* dst = reinterpret_cast<uint4*>(a.o + (orow * a.ld_o + (int64_t)qh * D + 32 * c) * 2);
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    uint32_t x[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[8 * g + 2 * e]) * inv_l,
                                                                       __uint_as_float(r[8 * g + 2 * e + 1]) * inv_l);
                        x[e] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    dst[g] = make_uint4(x[0], x[1], x[2], x[3]);
                }
            }
        }
        // O read before the next unit's first product overwrites it
        tc_fence_before();
    }
}

// ---- the issuing thread ----------------------------------------------------
// Per unit: QK_A(0), QK_B(0), then per key tile j: PV_A(j), QK_A(j+1), PV_B(j),
// QK_B(j+1).  The hazards:
//  - QK_X(j+1) overwrites S_X: issued only after p_full[X] of tile j;
//  - K is single-buffered: k_empty is committed after the tile's last Q K^T;
//  - softmax X(j) writes P_X and may rescale O_X once s_full[X](j) has fired,
//    which covers PV_X(j-1), issued before QK_X(j);
//  - V buffer b is released (v_empty) after the tile's last P V product;
//  - a unit's first products overwrite S_X, Q_X and O_X: q_full[X] of the unit
//    is signalled after softmax X has read the last unit's O_X.
template <int D>
__device__ __forceinline__ void mma_role(const AttnArgs& a, Shared& sh, uint32_t smem0, uint32_t tmem, Run run) {
    constexpr uint32_t ID_QK = idesc(0, kTile), ID_PV = idesc(1, D);
    auto qk = [&](int X) {
        const uint32_t q_s = smem0 + Smem<D>::q + X * Smem<D>::kOperand, k_s = smem0 + Smem<D>::k;
#pragma unroll
        for (int k = 0; k < D / 16; k++)
            mma_f16(tmem + kSCol + 128 * X, smem_desc(q_s + k * 4096, 2048, 128, kLayoutNone),
                    smem_desc(k_s + k * 4096, 2048, 128, kLayoutNone), ID_QK, k > 0);
        tc_commit(&sh.s_full[X]);
    };
    auto pv = [&](int X, uint32_t vb, bool acc) {
        const uint32_t p_s = smem0 + Smem<D>::p + X * Smem<D>::kP, v_s = smem0 + Smem<D>::v + vb * Smem<D>::kOperand;
#pragma unroll
        for (int k = 0; k < kTile / 16; k++)
            mma_f16(tmem + kOCol + 128 * X, smem_desc(p_s + k * 4096, 2048, 128, kLayoutNone),
                    smem_desc(v_s + k * 256, 128, 2048, kLayoutNone), ID_PV, (acc || k > 0) ? 1u : 0u);
    };
    int4 cut = make_int4(0, 0, 0, 0);
    uint32_t ph_q[2] = {0u, 0u}, ph_p[2] = {0u, 0u}, ph_k = 0u, nv = 0u;
    bool ok = true;
    Piece w;
    while (ok && next_piece<kChunkRows, kTile>(a, run, w)) {
        if (w.pieces) cut = make_int4(w.pieces, w.pair, w.head, 0);
        if (w.begin >= w.end) continue;
        const bool has_b = w.rows.n > kTile;
        if (!wait_or_stop(&sh.q_full[0], ph_q[0], sh, a, 6)) break;
        ph_q[0] ^= 1u;
        if (has_b) {
            if (!wait_or_stop(&sh.q_full[1], ph_q[1], sh, a, 6)) break;
            ph_q[1] ^= 1u;
        }
        if (!wait_or_stop(&sh.k_full, ph_k, sh, a, 7)) break;
        ph_k ^= 1u;
        tc_fence_after();
        qk(0);
        if (has_b) qk(1);
        tc_commit(&sh.k_empty);
        for (int i = w.begin; i < w.end; i++) {
            const bool more = i + 1 < w.end;
            const uint32_t vb = nv & 1u;
            if (!wait_or_stop(&sh.v_full[vb], (nv >> 1) & 1u, sh, a, 8) ||
                !wait_or_stop(&sh.p_full[0], ph_p[0], sh, a, 9)) {
                ok = false;
                break;
            }
            ph_p[0] ^= 1u;
            tc_fence_after();
            pv(0, vb, i > w.begin);
            if (more) {
                if (!wait_or_stop(&sh.k_full, ph_k, sh, a, 7)) {
                    ok = false;
                    break;
                }
                ph_k ^= 1u;
                tc_fence_after();
                qk(0);
            } else {
                tc_commit(&sh.o_full[0]);
            }
            if (has_b) {
                if (!wait_or_stop(&sh.p_full[1], ph_p[1], sh, a, 9)) {
                    ok = false;
                    break;
                }
                ph_p[1] ^= 1u;
                tc_fence_after();
                pv(1, vb, i > w.begin);
            }
            tc_commit(&sh.v_empty[vb]);
            nv++;
            if (more) {
                if (has_b) qk(1);
                tc_commit(&sh.k_empty);
            } else if (has_b) {
                tc_commit(&sh.o_full[1]);
            }
        }
    }
    a.cut[blockIdx.x] = cut;
    // every product issued is done before the TMEM is released (also after a stop)
    tc_commit(&sh.done);
    volatile int never = 0;
    if (!mbar_wait_bounded(&sh.done, 0, &never, kLimitNs)) record_error(a.v.err, NVFP4_ERR_TIMEOUT, 10);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Shared sh;
    RunScratch<kThreads>& scratch = *reinterpret_cast<RunScratch<kThreads>*>(smem);  // before the operands are there
    const int warp = threadIdx.x >> 5;
    const Run run = make_run<kChunkRows, kTile, kThreads, 1>(a, 0, kChunkLeast, scratch);
    if (threadIdx.x == 0) {
        for (int X = 0; X < 2; X++) {
            mbar_init(&sh.q_full[X], kSoft);
            mbar_init(&sh.s_full[X], 1);
            mbar_init(&sh.p_full[X], kSoft);
            mbar_init(&sh.o_full[X], 1);
            mbar_init(&sh.v_full[X], kProducers);
            mbar_init(&sh.v_empty[X], 1);
        }
        mbar_init(&sh.k_full, kProducers);
        mbar_init(&sh.k_empty, 1);
        mbar_init(&sh.done, 1);
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
    } else if (threadIdx.x == kMmaWarp * 32) {
        mma_role<D>(a, sh, smem0, tmem, run);
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
    chunk_kernel<D><<<ctas, kThreads, Smem<D>::bytes, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace

nvfp4_status launch_chunks(const AttnArgs& a, unsigned ctas, cudaStream_t stream) {
    return a.v.d == 128 ? launch<128>(a, ctas, stream) : launch<64>(a, ctas, stream);
}

}  // namespace paged
}  // namespace nvfp4
