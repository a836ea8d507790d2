// Matrix-vector products with an NVFP4 weight: y = ep(a32 * x W^T) for 1..16
// rows of bf16 activations x that are not quantized (the reading note's 4-bit
// weights, section 二 推理底座, for the few rows of a token-by-token step, where
// the W4A4 GEMM's 128-row tiles would stand empty).
//
// What bounds it: the weight is read once, 9/16 byte an element, and each
// element is used for at most 16 rows, so the weight's bytes are the floor and
// the work beside them is turning E2M1 codes and E4M3 scales into operands.
//
// One CTA an SM takes an equal share of the weight's groups of 16 rows.  Four
// groups {32 i + 16 half + 0..15} of a 128-row scale tile make a quad: the tile
// layout has the scales of four such rows in 16 consecutive bytes.  The warps
// split K in chunks of 128 columns and take three or four quads of rows at a
// time (a pass), so that a chunk's activations serve up to 256 rows.  The
// weight's bytes pass through a ring of (quad, chunk) pieces in shared memory a
// warp, which runs on across passes: 70 to 110 KB an SM on the way, and no
// registers wait.
// In a piece lane (g, t) reads 16 bytes (32 consecutive columns, two scale
// blocks) of rows g and g + 8 of each group; the columns of the 16 x 8 x 16
// matrix instruction are permuted so that these are its own A fragments, and
// the B fragments are 32 consecutive activations of row g.
//
// Operands: e2m1 * s is exact in binary16 (at most 6 significant bits); a row
// of activations is scaled by a power of two and rounded to binary16
// (fp4mma.cuh).  When all of them fit, the scaled activations lie in shared
// memory and the power comes off at the end; else a chunk's activations pass
// through the ring before its pieces and have a power of their own, which comes
// off the chunk's sums.
//
// Measured (here and below: no epilogue, calls in a graph, weights read from
// DRAM): 28672 x 8192 (132 MB) 31 us with one row (4.2 TB/s), 40 with 8, 49
// with 16; 14336 x 4096 12.4, 13.9, 17.7.  What bounds it is the conversion and
// integer pipe, with the issue slots half full: decoding a pair of codes takes
// 3.6 cycles of a scheduler, which alone is 14 us of that weight, and scaling the
// activations, addresses and scale bytes the rest; hence few, large passes.
// Measured and not taken, 16 rows of that weight: decoding into tensor memory as
// the A operand of tcgen05 products (97 us: 61 cycles a 128 x 16 x 16 product, and
// the pieces' addresses a lane), 12 warps and two quads a pass (52), pairs of
// groups interleaved there (56; with one row of eight it gains: 35 -> 32).
#include <cstdint>

#include "fp4mma.cuh"

namespace nvfp4 {
namespace gemv {

using namespace fp4mma;

constexpr int kSms = 148;
constexpr int kChunk = 128;  // columns of a piece
constexpr int kPiece = 64 * 64 + 2 * 16 * 16;  // a piece's codes, then its scales
constexpr int kMaxM = 16;
constexpr int kPitch = 64 + 4;  // of the partial sums' rows: the fragment stores spread over all banks

// Up to 8 rows (NT = 1): 16 warps of 128 registers, three quads a pass, two
// pieces a ring; up to 16 rows: 8 warps of 255, four quads, four pieces, since
// scaling a chunk's activations costs as much as a quad's products and is done
// once a pass (14336 x 4096, 16 rows: 21 -> 19 us against 12 warps and two quads).
template <int NT>
struct Cfg {
    static constexpr int kWarps = NT == 1 ? 16 : 8, kThreads = kWarps * 32, kStages = NT == 1 ? 2 : 4;
    static constexpr int kQuads = NT == 1 ? 3 : 4;  // of a pass
    static constexpr int kRing = kWarps * kStages * kPiece, kPart = kWarps * 8 * NT * kPitch * 4;
    static constexpr int kX = 227 * 1024 - 256 - kRing - kPart;  // what is left for activations
};

// A number known when compiling, as an argument.
template <int N>
struct Int {
    static constexpr int value = N;
};

struct Args {
    const uint8_t* x;  // bf16 [m][ldx]
    const uint8_t* codes;
    const uint8_t* scales;
    const float* a32;
    __nv_bfloat16* y;
    float* y32;
    const __nv_bfloat16 *bias, *mod_scale, *mod_shift, *gate, *residual;
    int64_t ldx, ldy, ld_res;
    int m, n, k, act;
    int chunks, groups;
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}

// What a CTA computes: `whole` quads from quad0 on, then the groups [g0, g1) of
// those that whole quads for every CTA leave over: one, an aligned pair or a
// quad, so that they lie in one quad (a piece's overhead is per quad).  Some CTAs
// then have less than others, or nothing; but dealt out evenly a share often lies
// in two quads.  One row, 16 rows (us; evenly):
//   4096 x 4096    6.2,  9.5  (8.0, 12.0)    9216 x 4096    8.2, 11.8  (9.9, 13.9)
//   5120 x 5120    8.5, 14.0 (10.3, 15.0)   14336 x 4096   12.4, 17.7 (13.3, 18.5)
//   6144 x 4096    7.7, 11.8  (9.0, 13.0)   28672 x 8192   31.2, 49.2 (31.4, 50.2)
// With 8 rows the wide ones lose by it: 20000 x 4096 17.1 (16.9), 28672 x 8192
// 40.4 (39.2).  The longest share stays above the mean (2.3 times at 1024 rows, 1.3
// at 14336): K is not split over CTAs.
struct Share {
    int quad0, whole, g0, g1;
    __device__ __forceinline__ int count() const { return whole + (g1 > g0 ? 1 : 0); }
};

// The CTA's q-th quad: of its rows 16 i + r, i in [lo, hi) belong to the CTA and
// are rows `row0` + 32 i + r of the weight.
struct Quad {
    int row0, lo, hi;
    __device__ __forceinline__ Quad(const Share& s, int i) {
        const bool full = i < s.whole;
        const int q = full ? s.quad0 + i : s.g0 / 4;
        row0 = (q >> 1) * 128 + (q & 1) * 16;
        lo = full ? 0 : s.g0 & 3;
        hi = full ? 4 : lo + s.g1 - s.g0;
    }
};

// The piece (quad, chunk c) into a ring slot; what lies outside the weight is
// zeros, and groups of other CTAs are not read.
__device__ __forceinline__ void load_piece(const Args& a, const Quad& q, int c, int lane, uint32_t dst) {
    const int64_t pitch = a.k / 2;
    const int part = lane & 3, r = lane >> 2, col = c * kChunk + 32 * part;
    const bool in_k = col < a.k;  // k is a multiple of 64, so the lane's 32 columns are in or out as a whole
    const uint8_t* p = a.codes + (int64_t)(q.row0 + r) * pitch + col / 2;
    const uint32_t d = dst + r * 64 + 16 * part;
    if (q.row0 + 112 <= a.n && (c + 1) * kChunk <= a.k) {
#pragma unroll
        for (int i = 0; i < 4; i++, p += 32 * pitch)
            if (i >= q.lo && i < q.hi) {
                copy16(d + 16 * i * 64, p, true);
                copy16(d + (16 * i + 8) * 64, p + 8 * pitch, true);
            }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i >= q.lo && i < q.hi) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int row = 32 * i + 8 * h;
                    const bool real = in_k && q.row0 + r + row < a.n;
                    copy16(d + (16 * i + 8 * h) * 64, real ? p + row * pitch : a.codes, real);
                }
            }
    }
    // two scale tiles (64 columns each), 16 rows of 16 bytes; the tiles cover rows up to the next multiple of 128
    const int tile = lane >> 4, tcol = c * kChunk + 64 * tile;
    const bool real = tcol < a.k;
    const uint8_t* ps = a.scales + ((int64_t)(q.row0 >> 7) * (a.k / 64) + tcol / 64) * 512 + ((q.row0 & 31) + (lane & 15)) * 16;
    copy16(dst + 64 * 64 + lane * 16, real ? ps : a.scales, real);
}

// Where 16-byte piece j (8 values) of a chunk's row r lies among the row's 16:
// the four lanes of two rows then read eight different bank groups.
__device__ __forceinline__ int x_place(int r, int j) { return (j & ~3) | ((j ^ (j >> 2) ^ (r & 1)) & 3); }

// A chunk's activations (bf16) into a ring slot, the pieces of a row placed as above; columns behind K are zeros.
__device__ __forceinline__ void load_x(const Args& a, int c, int lane, uint32_t dst) {
    const int r = lane >> 4, j = lane & 15, col = c * kChunk + 8 * j;
    const bool real = col < a.k;
    const uint8_t* p = a.x + ((int64_t)r * a.ldx + (real ? col : 0)) * 2;
    const uint32_t d = dst + r * 256 + x_place(r, j) * 16;  // (rows 2 on: the same place)
    for (int m = 0; m + r < a.m; m += 2, p += a.ldx * 4) copy16(d + m * 256, p, real);
}

// 32 codes of one row with their two block scales -> 16 operand pairs
__device__ __forceinline__ void decode32(const uint4& c, uint32_t two_scales, uint32_t* o) {
    const __half2 s = e4m3x2_to_half2((uint16_t)two_scales);
    const __half2 s0 = __low2half2(s), s1 = __high2half2(s);
    decode8(c.x, s0, o);
    decode8(c.y, s0, o + 4);
    decode8(c.z, s1, o + 8);
    decode8(c.w, s1, o + 12);
}

__device__ __forceinline__ float act_gelu(float y) {
    const float u = 0.7978845608028654f * (y + 0.044715f * y * y * y);  // sqrt(2 / pi)
    return 0.5f * y * (1.0f + tanhf(u));
}

template <int NT, bool XS>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, 1) gemv_kernel(const __grid_constant__ Args a) {
    constexpr int kWarps = Cfg<NT>::kWarps, kThreads = Cfg<NT>::kThreads, kStages = Cfg<NT>::kStages, kQuads = Cfg<NT>::kQuads;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t row_max[kMaxM];
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kStages * kPiece);
    float(*part)[8 * NT][kPitch] = reinterpret_cast<float(*)[8 * NT][kPitch]>(smem + Cfg<NT>::kRing);
    const uint32_t xs = smem_u32(smem) + Cfg<NT>::kRing + Cfg<NT>::kPart;
    if (threadIdx.x < kMaxM) row_max[threadIdx.x] = 0u;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Share share;
    share.whole = a.groups / 4 / (int)gridDim.x;
    share.quad0 = share.whole * (int)blockIdx.x;
    const int spread = share.whole * (int)gridDim.x * 4, rest = a.groups - spread;  // rest < 4 gridDim.x
    const int each = rest <= (int)gridDim.x ? 1 : rest <= 2 * (int)gridDim.x ? 2 : 4;
    share.g0 = min(a.groups, spread + each * (int)blockIdx.x);
    share.g1 = min(a.groups, share.g0 + each);
    const int quads = share.count();
    if (quads == 0) return;

    // the next piece to fetch: pass by pass, chunk by chunk, (the chunk's activations, then) quad by quad
    constexpr int kBefore = XS ? 0 : 1;
    int f_quad = -kBefore, f_pass = 0, f_chunk = warp, f_slot = 0;
    auto fetch = [&]() {
        if (f_chunk < a.chunks && f_pass < quads) {
            if (!XS && f_quad < f_pass) load_x(a, f_chunk, lane, ring + (uint32_t)(f_slot * kPiece));
            else load_piece(a, Quad(share, f_quad), f_chunk, lane, ring + (uint32_t)(f_slot * kPiece));
            f_slot = f_slot == kStages - 1 ? 0 : f_slot + 1;
            if (++f_quad >= min(quads, f_pass + kQuads)) {
                f_chunk += kWarps;
                if (f_chunk >= a.chunks) {
                    f_chunk = warp;
                    f_pass += kQuads;
                }
                f_quad = f_pass - kBefore;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) fetch();

    float down[NT][2];  // what the sums' columns 2t, 2t + 1 are multiplied by
    if (XS) {
        // the rows' largest magnitudes, then the scaled rows; a thread keeps what it has read (a warp has whole rows'
        // parts, of 32 x 8 activations, so that its maximum is one row's)
        constexpr int kParts = (Cfg<NT>::kX / 16 + kThreads - 1) / kThreads + 1;
        const int row_parts = (a.chunks * 16 + 31) / 32, parts = row_parts * a.m;
        uint4 v[kParts];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kParts; i++) {
            const int p = warp + i * kWarps, m = p / row_parts, j = (p - m * row_parts) * 32 + lane;
            v[i] = p < parts && j < a.k / 8 ? ld_coherent(reinterpret_cast<const uint4*>(a.x + (int64_t)m * a.ldx * 2) + j)
                                            : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kParts; i++) {
            const int p = warp + i * kWarps;
            if (p >= parts) break;
            const uint32_t mx = __reduce_max_sync(0xFFFFFFFFu, max_bits<1>(&v[i]));
            if (lane == 0) atomicMax(&row_max[p / row_parts], mx);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int e = 0; e < 2; e++) down[j][e] = row_scale(row_max[8 * j + 2 * t + e]).down;
#pragma unroll
        for (int i = 0; i < kParts; i++) {
            const int p = warp + i * kWarps, m = p / row_parts, j = (p - m * row_parts) * 32 + lane;
            if (p >= parts) break;
            if (j < a.chunks * 16) {
                uint32_t h[4];
                scale8(v[i], row_scale(row_max[m]).up, h);
                st_shared16(xs + ((j >> 4) * a.m + m) * 256 + x_place(m, j & 15) * 16, make_uint4(h[0], h[1], h[2], h[3]));
            }
        }
        __syncthreads();
    }

    const float alpha = ld_coherent(a.a32);
    int slot = 0;
    auto next_piece = [&]() {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();  // the piece is there for every lane, and every lane has left the slot that is filled next
        fetch();
        const uint32_t at = ring + (uint32_t)(slot * kPiece);
        slot = slot == kStages - 1 ? 0 : slot + 1;
        return at;
    };
    for (int pass = 0; pass < quads; pass += kQuads) {
        float acc[kQuads][NT][4][4];
#pragma unroll
        for (int q = 0; q < kQuads; q++)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[q][j][i][e] = 0.0f;
#pragma unroll 1
        for (int c = warp; c < a.chunks; c += kWarps) {
            // (columns of the product that are no row of x hold anything: nobody reads them)
            uint32_t xb[NT][16], px = xs + c * a.m * 256;
            if (!XS) px = next_piece();
#pragma unroll
            for (int j = 0; j < NT; j++) {
                const int m = min(8 * j + g, a.m - 1);
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    v[i] = lds16(px + m * 256 + x_place(m, 4 * t + i) * 16);
                    if (XS) xb[j][4 * i] = v[i].x, xb[j][4 * i + 1] = v[i].y, xb[j][4 * i + 2] = v[i].z, xb[j][4 * i + 3] = v[i].w;
                }
                if (!XS) {  // a scale for the chunk; columns 2t, 2t + 1 are rows of lanes (2t, .), (2t + 1, .)
                    const float back = scale_row<4>(v, xb[j]);
                    down[j][0] = __shfl_sync(0xFFFFFFFFu, back, 8 * t);
                    down[j][1] = __shfl_sync(0xFFFFFFFFu, back, 8 * t + 4);
                }
            }
#pragma unroll
            for (int q = 0; q < kQuads; q++) {
                if (pass + q >= quads) continue;
                const Quad quad(share, pass + q);
                const uint32_t at = next_piece();
                const uint32_t scales = at + 64 * 64 + (t >> 1) * 256 + g * 16, codes = at + g * 64 + 16 * t;
                const uint4 s0 = lds16(scales), s1 = lds16(scales + 8 * 16);
                const int sh = 16 * (t & 1);
                const uint32_t sc[4][2] = {
                    {s0.x >> sh, s1.x >> sh}, {s0.y >> sh, s1.y >> sh}, {s0.z >> sh, s1.z >> sh}, {s0.w >> sh, s1.w >> sh}};
                // groups first .. first + number - 1, interleaved so that no product waits for the one before it
                auto groups = [&](auto first, auto number) {
                    constexpr int i0 = decltype(first)::value, n = decltype(number)::value;
                    uint4 c[n][2];
                    __half2 s[n][2];
                    float chunk[XS ? 1 : n][NT][4];
#pragma unroll
                    for (int i = 0; i < n; i++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            c[i][h] = lds16(codes + (16 * (i0 + i) + 8 * h) * 64);
                            s[i][h] = e4m3x2_to_half2((uint16_t)sc[i0 + i][h]);
                        }
#pragma unroll
                    for (int w = 0; w < 4; w++)
#pragma unroll
                        for (int i = 0; i < n; i++) {
                            uint32_t w0[4], w1[4];
                            auto word = [&](const uint4& v) { return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w; };
                            decode8(word(c[i][0]), w < 2 ? __low2half2(s[i][0]) : __high2half2(s[i][0]), w0);
                            decode8(word(c[i][1]), w < 2 ? __low2half2(s[i][1]) : __high2half2(s[i][1]), w1);
#pragma unroll
                            for (int e = 0; e < 2; e++)
#pragma unroll
                                for (int j = 0; j < NT; j++) {
                                    float* d = XS ? acc[q][j][i0 + i] : chunk[XS ? 0 : i][j];
                                    const uint32_t b0 = xb[j][4 * w + 2 * e], b1 = xb[j][4 * w + 2 * e + 1];
                                    if (!XS && w == 0 && e == 0) mma_16816_first(d, w0[0], w1[0], w0[1], w1[1], b0, b1);
                                    else mma_16816(d, w0[2 * e], w1[2 * e], w0[2 * e + 1], w1[2 * e + 1], b0, b1);
                                }
                        }
                    if (!XS)
#pragma unroll
                        for (int i = 0; i < n; i++)
#pragma unroll
                            for (int j = 0; j < NT; j++)
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    acc[q][j][i0 + i][e] = fmaf(chunk[XS ? 0 : i][j][e], down[j][e & 1], acc[q][j][i0 + i][e]);
                };
                if (NT == 1 && quad.lo == 0 && quad.hi == 4) {
                    groups(Int<0>{}, Int<4>{});
                } else {
                    if (quad.lo <= 0 && quad.hi > 0) groups(Int<0>{}, Int<1>{});
                    if (quad.lo <= 1 && quad.hi > 1) groups(Int<1>{}, Int<1>{});
                    if (quad.lo <= 2 && quad.hi > 2) groups(Int<2>{}, Int<1>{});
                    if (quad.lo <= 3 && quad.hi > 3) groups(Int<3>{}, Int<1>{});
                }
            }
        }
        // the warps' sums, in a fixed order, and the epilogue
#pragma unroll
        for (int q = 0; q < kQuads; q++) {
            if (pass + q >= quads) continue;
            const Quad quad(share, pass + q);
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        part[warp][8 * j + 2 * t + (e & 1)][16 * i + g + 8 * (e >> 1)] =
                            XS ? acc[q][j][i][e] * down[j][e & 1] : acc[q][j][i][e];
            __syncthreads();
            for (int o = threadIdx.x; o < a.m * 64; o += kThreads) {
                const int m = o / 64, r = o % 64;
                const int n = quad.row0 + (r >> 4) * 32 + (r & 15);
                if ((r >> 4) < quad.lo || (r >> 4) >= quad.hi || n >= a.n) continue;
                float s = part[0][m][r];
#pragma unroll
                for (int w = 1; w < kWarps; w++) s += part[w][m][r];
                float y = a.bias ? fmaf(alpha, s, __bfloat162float(a.bias[n])) : alpha * s;
                if (a.act == NVFP4_ACT_GELU_TANH) y = act_gelu(y);
                if (a.mod_scale) y = __fmul_rn(y, __fadd_rn(1.0f, __bfloat162float(a.mod_scale[n])));
                if (a.mod_shift) y = __fadd_rn(y, __bfloat162float(a.mod_shift[n]));
                if (a.gate) y = __fmul_rn(__bfloat162float(a.gate[n]), y);
                if (a.residual) y = __fadd_rn(__bfloat162float(a.residual[(int64_t)m * a.ld_res + n]), y);
                if (a.y) a.y[(int64_t)m * a.ldy + n] = __float2bfloat16_rn(y);
                if (a.y32) a.y32[(int64_t)m * a.n + n] = y;
            }
            __syncthreads();
        }
    }
}

}  // namespace gemv
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_gemv(const void* x_bf16, int64_t m, int64_t ldx, const nvfp4_tensor* W, void* y_bf16,
                                   int64_t ldy, const nvfp4_epilogue* ep, nvfp4_stream_t stream) {
    if (!W || !W->codes || !W->scales || !W->global_scale || m < 0 || W->rows <= 0 || W->cols <= 0)
        return NVFP4_ERR_INVALID_ARG;
    const int64_t n = W->rows, k = W->cols;
    if (k % 64 != 0 || n > (1 << 30) || k > (1 << 30) || m > gemv::kMaxM) return NVFP4_ERR_UNSUPPORTED;
    float* y32 = ep ? ep->debug_y : nullptr;
    if (ldx < k || (y_bf16 && ldy < n)) return NVFP4_ERR_INVALID_ARG;
    if (ep) {
        if (ep->act != NVFP4_ACT_NONE && ep->act != NVFP4_ACT_GELU_TANH) return NVFP4_ERR_INVALID_ARG;
        if (ep->debug_flags) return NVFP4_ERR_INVALID_ARG;
        if (ep->residual && ep->ld_residual < n) return NVFP4_ERR_INVALID_ARG;
        if (ep->out_codes || ep->out_scales || ep->out_global_scale || ep->out_amax || ep->out_col0 || ep->out_cols)
            return NVFP4_ERR_UNSUPPORTED;
    }
    if (m == 0) return NVFP4_OK;  // (before the row tensors: an empty one has no address)
    if (!x_bf16 || (!y_bf16 && !y32)) return NVFP4_ERR_INVALID_ARG;
    auto odd = [](const void* p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
    if (odd(x_bf16, 15u) || ldx % 8 != 0 || odd(W->codes, 15u) || odd(W->scales, 15u) || odd(W->global_scale, 3u) ||
        odd(y_bf16, 1u) || odd(y32, 3u))
        return NVFP4_ERR_MISALIGNED;
    gemv::Args a{};
    if (ep) {
        const void* vecs[5] = {ep->bias, ep->mod_scale, ep->mod_shift, ep->gate, ep->residual};
        for (const void* v : vecs)
            if (odd(v, 1u)) return NVFP4_ERR_MISALIGNED;
        a.bias = static_cast<const __nv_bfloat16*>(ep->bias);
        a.mod_scale = static_cast<const __nv_bfloat16*>(ep->mod_scale);
        a.mod_shift = static_cast<const __nv_bfloat16*>(ep->mod_shift);
        a.gate = static_cast<const __nv_bfloat16*>(ep->gate);
        a.residual = static_cast<const __nv_bfloat16*>(ep->residual);
        a.ld_res = ep->ld_residual;
        a.act = ep->act;
    }
    a.x = static_cast<const uint8_t*>(x_bf16);
    a.codes = static_cast<const uint8_t*>(W->codes);
    a.scales = static_cast<const uint8_t*>(W->scales);
    a.a32 = W->global_scale;
    a.y = static_cast<__nv_bfloat16*>(y_bf16);
    a.y32 = y32;
    a.ldx = ldx;
    a.ldy = ldy;
    a.m = (int)m;
    a.n = (int)n;
    a.k = (int)k;
    a.chunks = (int)((k + gemv::kChunk - 1) / gemv::kChunk);
    // groups of 16 rows, eight a 128-row scale tile (the last tile's may be padding)
    a.groups = (int)((n + 127) / 128 * 8);
    static PerDevice<int> ready;
    int done = 0;
    const nvfp4_status st = ready.get(&done, [](int, int& v) {
        v = 1;
        const void* kernels[4] = {(const void*)gemv::gemv_kernel<1, false>, (const void*)gemv::gemv_kernel<1, true>,
                                  (const void*)gemv::gemv_kernel<2, false>, (const void*)gemv::gemv_kernel<2, true>};
        for (const void* f : kernels)
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 256) != cudaSuccess)
                return NVFP4_ERR_CUDA;
        return NVFP4_OK;
    });
    if (st != NVFP4_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.groups < gemv::kSms ? a.groups : gemv::kSms));
    const bool two = m > 8;
    const int64_t xbytes = (int64_t)a.chunks * m * 256, room = two ? gemv::Cfg<2>::kX : gemv::Cfg<1>::kX;
    const bool xs = xbytes <= room;  // (then at most 102 or 106 parts, of the 128 or 112 that the warps hold)
    cfg.blockDim = dim3((unsigned)(two ? gemv::Cfg<2>::kThreads : gemv::Cfg<1>::kThreads));
    cfg.dynamicSmemBytes = (size_t)((two ? gemv::Cfg<2>::kRing + gemv::Cfg<2>::kPart
                                         : gemv::Cfg<1>::kRing + gemv::Cfg<1>::kPart) + (xs ? xbytes : 0));
    cfg.stream = (cudaStream_t)stream;
    // programmatic dependent launch: the grid's start overlaps the previous kernel's end (the kernel waits for it
    // before it reads anything)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg,
                           two ? (xs ? gemv::gemv_kernel<2, true> : gemv::gemv_kernel<2, false>)
                               : (xs ? gemv::gemv_kernel<1, true> : gemv::gemv_kernel<1, false>),
                           a) != cudaSuccess) {
        cudaGetLastError();
        return NVFP4_ERR_CUDA;
    }
    return NVFP4_OK;
}
