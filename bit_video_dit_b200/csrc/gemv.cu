// Matrix-vector products with an NVFP4 weight: y = ep(a32 * x W^T) for 1..16
// rows of bf16 activations x that are not quantized (the reading note's 4-bit
// weights, section 二 推理底座, for the few rows of a token-by-token step, where
// the W4A4 GEMM's 128-row tiles would stand empty).
//
// What bounds it: the weight is read once, 9/16 byte an element, and each
// element is used for at most 16 rows, so the weight's bytes are the floor and
// the work beside them is turning E2M1 codes and E4M3 scales into operands.
//
// One CTA (8 warps) takes the 64 weight rows {32 i + 16 half + 0..15} of a
// 128-row scale tile: there the tile layout puts the four scales of four such
// rows into 16 consecutive bytes, so one 16-byte load serves four row groups.
// The warps (and the CTAs of a cluster) split K in chunks of 128 columns.  In
// a chunk lane (g, t) loads 16 bytes (32 consecutive columns, two scale
// blocks) of rows g and g + 8 of each row group; the columns of the 16 x 8 x 16
// matrix instruction are permuted so that these are its own A fragments, and
// the B fragments are 32 consecutive activations of row g.
//
// Operands: e2m1 * s is exact in binary16 (at most 6 significant bits); a row
// of activations is scaled by a power of two per chunk and rounded to binary16
// (fp4mma.cuh), and the power comes off in the binary32 accumulation over the
// chunks.
#include <cstdint>

#include "fp4mma.cuh"

namespace nvfp4 {
namespace gemv {

using namespace fp4mma;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 64;         // weight rows of a CTA
constexpr int kChunk = 128;       // columns a warp takes at a time
constexpr int kMaxM = 16;
constexpr int kPitch = kRows + 4;  // of the partial sums' rows: the fragment stores spread over all banks

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
    int chunks, cluster;
};

// The chunk's weight bytes and activations of one lane.
template <int NT>
struct Loaded {
    uint4 c[8];      // codes of rows 32 i + g and 32 i + g + 8, i = 0..3
    uint4 s[2];      // scale bytes of the rows' tile: word i belongs to row group i
    uint4 x[NT][4];  // 32 activations of row g of each row tile
};

template <int NT>
__device__ __forceinline__ void load_chunk(const Args& a, int row0, int c, int g, int t, Loaded<NT>& l) {
    const int col = c * kChunk + 32 * t;
    const bool in_k = col < a.k;  // k is a multiple of 64, so the lane's 32 columns are in or out as a whole
    const int64_t pitch = a.k / 2;
    const uint8_t* p = a.codes + (int64_t)(row0 + g) * pitch + col / 2;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int r = (i >> 1) * 32 + (i & 1) * 8;
        l.c[i] = in_k && row0 + g + r < a.n ? ld_stream16(p + r * pitch) : make_uint4(0u, 0u, 0u, 0u);
    }
    // tile (row0 / 128, col / 64); the tiles cover rows up to the next multiple of 128
    const uint8_t* ps = a.scales + ((int64_t)(row0 >> 7) * (a.k / 64) + col / 64) * 512 + ((row0 & 31) + g) * 16;
#pragma unroll
    for (int h = 0; h < 2; h++) l.s[h] = in_k ? ld_stream16(ps + 128 * h) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < NT; j++) {
        const uint4* px = reinterpret_cast<const uint4*>(a.x + ((int64_t)(8 * j + g) * a.ldx + col) * 2);
#pragma unroll
        for (int i = 0; i < 4; i++)
            l.x[j][i] = in_k && 8 * j + g < a.m ? __ldg(px + i) : make_uint4(0u, 0u, 0u, 0u);
    }
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

__device__ __forceinline__ float peer_f32(const float* p, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(p), rank)));
    return v;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) gemv_kernel(const __grid_constant__ Args a) {
    __shared__ float part[kWarps][8 * NT][kPitch];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rank = a.cluster == 1 ? 0 : (int)(blockIdx.x % (unsigned)a.cluster);
    const int tile = (int)(blockIdx.x / (unsigned)a.cluster);
    const int row0 = (tile >> 1) * 128 + (tile & 1) * 16;  // rows row0 + 32 i + 0..15
    float acc[NT][4][4];
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[j][i][e] = 0.0f;

    const int step = kWarps * a.cluster;
    for (int c = rank * kWarps + warp; c < a.chunks; c += step) {
        Loaded<NT> l;
        load_chunk<NT>(a, row0, c, g, t, l);
        uint32_t xb[NT][16];
        float inv[NT][2];
#pragma unroll
        for (int j = 0; j < NT; j++) {
            const float back = scale_row<4>(l.x[j], xb[j]);
            // the fragment's columns 2t, 2t + 1 are activation rows held by lanes (2t, .), (2t + 1, .)
            inv[j][0] = __shfl_sync(0xFFFFFFFFu, back, 8 * t);
            inv[j][1] = __shfl_sync(0xFFFFFFFFu, back, 8 * t + 4);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t s0 = i == 0 ? l.s[0].x : i == 1 ? l.s[0].y : i == 2 ? l.s[0].z : l.s[0].w;
            const uint32_t s1 = i == 0 ? l.s[1].x : i == 1 ? l.s[1].y : i == 2 ? l.s[1].z : l.s[1].w;
            uint32_t w0[16], w1[16];
            decode32(l.c[2 * i], s0 >> (16 * (t & 1)), w0);
            decode32(l.c[2 * i + 1], s1 >> (16 * (t & 1)), w1);
#pragma unroll
            for (int j = 0; j < NT; j++) {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < 8; e++)
                    mma_16816(d, w0[2 * e], w1[2 * e], w0[2 * e + 1], w1[2 * e + 1], xb[j][2 * e], xb[j][2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 4; e++) acc[j][i][e] = fmaf(d[e], inv[j][e & 1], acc[j][i][e]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                part[warp][8 * j + 2 * t + (e & 1)][16 * i + g + 8 * (e >> 1)] = acc[j][i][e];
    __syncthreads();
    // the warps' sums, then the cluster's, in a fixed order
    const int outs = a.m * kRows;
    if (a.cluster > 1) {
        for (int o = threadIdx.x; o < outs; o += kThreads) {
            const int n = o / kRows, r = o % kRows;
            float s = part[0][n][r];
#pragma unroll
            for (int w = 1; w < kWarps; w++) s += part[w][n][r];
            part[0][n][r] = s;
        }
        cluster_sync_all();
    }
    const float alpha = __ldg(a.a32);
    const int share = (outs + a.cluster - 1) / a.cluster;
    const int last = min(outs, (rank + 1) * share);
    for (int o = rank * share + threadIdx.x; o < last; o += kThreads) {
        const int m = o / kRows, r = o % kRows;
        const int n = row0 + (r >> 4) * 32 + (r & 15);
        float s = 0.0f;
        if (a.cluster > 1) {
            for (int q = 0; q < a.cluster; q++) s += peer_f32(&part[0][m][r], (uint32_t)q);
        } else {
#pragma unroll
            for (int w = 0; w < kWarps; w++) s += part[w][m][r];
        }
        if (n >= a.n) continue;
        float y = a.bias ? fmaf(alpha, s, __bfloat162float(a.bias[n])) : alpha * s;
        if (a.act == NVFP4_ACT_GELU_TANH) y = act_gelu(y);
        if (a.mod_scale) y = __fmul_rn(y, __fadd_rn(1.0f, __bfloat162float(a.mod_scale[n])));
        if (a.mod_shift) y = __fadd_rn(y, __bfloat162float(a.mod_shift[n]));
        if (a.gate) y = __fmul_rn(__bfloat162float(a.gate[n]), y);
        if (a.residual) y = __fadd_rn(__bfloat162float(a.residual[(int64_t)m * a.ld_res + n]), y);
        if (a.y) a.y[(int64_t)m * a.ldy + n] = __float2bfloat16_rn(y);
        if (a.y32) a.y32[(int64_t)m * a.n + n] = y;
    }
    // a CTA's shared memory stays until every peer has read it
    if (a.cluster > 1) cluster_sync_all();
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
    if (!y_bf16 && !y32) return NVFP4_ERR_INVALID_ARG;
    if (ldx < k || (y_bf16 && ldy < n)) return NVFP4_ERR_INVALID_ARG;
    if (ep) {
        if (ep->act != NVFP4_ACT_NONE && ep->act != NVFP4_ACT_GELU_TANH) return NVFP4_ERR_INVALID_ARG;
        if (ep->debug_flags) return NVFP4_ERR_INVALID_ARG;
        if (ep->residual && ep->ld_residual < n) return NVFP4_ERR_INVALID_ARG;
        if (ep->out_codes || ep->out_scales || ep->out_global_scale || ep->out_amax || ep->out_col0 || ep->out_cols)
            return NVFP4_ERR_UNSUPPORTED;
    }
    if (m == 0) return NVFP4_OK;
    if (!x_bf16) return NVFP4_ERR_INVALID_ARG;
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
    // 64-row tiles: two a 128-row block (the second of the last block may be all padding rows)
    const int64_t tiles = (n + 127) / 128 * 2;
    // K is split over a cluster until two CTAs an SM (148 SMs) have work, as long as every warp keeps a chunk
    a.cluster = 1;
    while (a.cluster < 8 && tiles * a.cluster < 2 * 148 && a.chunks >= 2 * a.cluster * gemv::kWarps) a.cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * a.cluster));
    cfg.blockDim = dim3(gemv::kThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, a.m <= 8 ? gemv::gemv_kernel<1> : gemv::gemv_kernel<2>, a) != cudaSuccess) {
        cudaGetLastError();
        return NVFP4_ERR_CUDA;
    }
    return NVFP4_OK;
}
