// E4M3 codes with one fp32 scale per 128 elements: rows of activations
// (1 x 128 along a row, the rows optionally gathered), token columns of each
// expert (128 x 1 down its rows, transposed output) and weights (128 x 128,
// both orientations).
//
// A block with maximum magnitude a: c = max(a, 2^-100), code of x =
// E4M3_RNE(RN(x * RN(448 / c))) (saturating: the product may round past 448),
// scale = RN(c / 448), and 0 for an all-zero block.  The two divisions are the
// IEEE ones, once per block; an element costs one multiply, one clamp and its
// share of a packed conversion, so every kernel here is bound by its bytes:
// 2 per element read, 1 or 2 written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsq.h"
#include "device_common.h"

namespace bsq {

constexpr float B128_TINY = 0x1p-100f;

struct B128Scale {
    float inv, scale;
};
// From the maximum's bf16 magnitude bits.
__device__ __forceinline__ B128Scale b128_scale(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits << 16);
    const float c = fmaxf(a, B128_TINY);
    return {448.0f / c, a > 0.0f ? c / 448.0f : 0.0f};
}

// E4M3 codes of four packed pairs (8 elements) times inv.
__device__ __forceinline__ uint2 b128_codes8(uint4 w, float inv) {
    return make_uint2(e4m3x4(bf16_lo(w.x) * inv, bf16_hi(w.x) * inv, bf16_lo(w.y) * inv, bf16_hi(w.y) * inv),
                      e4m3x4(bf16_lo(w.z) * inv, bf16_hi(w.z) * inv, bf16_lo(w.w) * inv, bf16_hi(w.w) * inv));
}

__device__ __forceinline__ uint32_t absmax8(uint4 w) {
    return fold_max16(absmax2_bf16(absmax2_bf16(absmax2_bf16(w.x & 0x7FFF7FFFu, w.y), w.z), w.w));
}

// Maximum over a group of 16 lanes.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 16));
    return v;
}

// Rows.  Sixteen lanes take a block (8 elements, 16 bytes each), a workgroup
// of 256 threads 16 rows x 8 blocks: its 16 groups run down the rows, so four
// rows of loads per wave are in flight for each of 8 steps along the row.
// Scales leave as runs of 16 rows (64 bytes of the block-major layout).
constexpr int ROWS_R = 16, ROWS_B = 8;
template <bool GATHER>
__global__ __launch_bounds__(256) void k_quantize_b128_rows(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                            int64_t ld, const int32_t* __restrict__ row_index,
                                                            int64_t src_rows, uint8_t* __restrict__ codes,
                                                            float* __restrict__ scale) {
    __shared__ float s_scale[ROWS_B][ROWS_R];
    const int g = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int64_t r = (int64_t)blockIdx.x * ROWS_R + g;
    const int b0 = blockIdx.y * ROWS_B;
    const int nb = (cols + 127) / 128;
    int64_t src = r < rows ? r : -1;
    if (GATHER && r < rows) {
        const int32_t i = row_index[r];
        src = (uint32_t)i < (uint64_t)src_rows ? i : -1;
    }
    uint4 w[ROWS_B];
#pragma unroll
    for (int b = 0; b < ROWS_B; ++b) {
        const int c = 128 * (b0 + b) + 8 * l;
        w[b] = make_uint4(0, 0, 0, 0);
        if (src >= 0 && c < cols) w[b] = *reinterpret_cast<const uint4*>(x + src * ld + c);
    }
#pragma unroll
    for (int b = 0; b < ROWS_B; ++b) {
        const int c = 128 * (b0 + b) + 8 * l;
        const B128Scale q = b128_scale(max16(absmax8(w[b])));
        if (l == 0) s_scale[b][g] = q.scale;
        if (r < rows && c < cols) *reinterpret_cast<uint2*>(codes + r * cols + c) = b128_codes8(w[b], q.inv);
    }
    __syncthreads();
    const int b = threadIdx.x >> 4;
    const int64_t rr = (int64_t)blockIdx.x * ROWS_R + l;
    if (b < ROWS_B && b0 + b < nb && rr < rows) scale[(int64_t)(b0 + b) * rows + rr] = s_scale[b][l];
}

// One 128 x 128 tile staged in LDS as bf16, 16-byte chunk c of row r at chunk
// position c ^ (r & 15): reads along a row and down a column pair both spread
// over the banks.
__device__ __forceinline__ uint32_t tile_at(int r, int chunk) { return (uint32_t)(r * 256 + 16 * (chunk ^ (r & 15))); }

// Pitch of the transposed codes in LDS: 33 dwords, so that 64 lanes writing one
// dword to rows two apart meet two to a bank, the rate of a 256-byte write.
constexpr int TILE_T = 132;

// Token columns of a group (and optionally the rows' own 1 x 128 codes): tile
// t of P/128 covers up to 128 rows of one group, tile column j 128 channels.
template <bool GATHER, bool ROWS>
__global__ __launch_bounds__(256) void k_quantize_b128_cols(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                            int64_t ld, const int32_t* __restrict__ row_index,
                                                            int64_t src_rows, const int32_t* __restrict__ offsets,
                                                            int G, int64_t P, uint8_t* __restrict__ codes,
                                                            float* __restrict__ scale, uint8_t* __restrict__ t_codes,
                                                            float* __restrict__ t_scale) {
    __shared__ __align__(16) uint8_t s_x[128 * 256];
    __shared__ uint32_t s_max[4][128];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t blk = blockIdx.y;
    const int c0 = blockIdx.x * 128;
    const int nc = min(128, cols - c0);
    // the group whose 128-column tiles hold this one: groups start at block
    // g + offsets[g] / 128, so the starts increase and the last one at or
    // before blk owns it if it has rows there.  The rows past the last group
    // are a group G of their own here, whose columns stay zero.
    int grp = 0;
    for (int base = 0; base <= G; base += 64) {
        const int g = base + lane;
        const int64_t st = g <= G ? g + (int64_t)max(0, offsets[g]) / 128 : (int64_t)1 << 40;
        const int n = __builtin_popcountll(__ballot(st <= blk));
        if (n > 0) grp = base + n - 1;
        if (n < 64) break;
    }
    const bool tail = grp == G;
    const int64_t o0 = offsets[grp], o1 = tail ? rows : min((int64_t)offsets[grp + 1], rows);
    const int64_t first = o0 + 128 * (blk - grp - max((int64_t)0, o0) / 128);
    const int nr = (o0 >= 0 && first >= o0) ? (int)max((int64_t)0, min((int64_t)128, o1 - first)) : 0;

    // load: 16 threads a row, 8 steps of 16 rows
    const bool need = ROWS || !tail;
    const int ch = tid & 15, rg = tid >> 4;
    uint4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 16 * i + rg;
        w[i] = make_uint4(0, 0, 0, 0);
        if (need && r < nr && 8 * ch < nc) {
            int64_t src = first + r;
            if (GATHER) {
                const int32_t k = row_index[src];
                src = (uint32_t)k < (uint64_t)src_rows ? k : -1;
            }
            if (src >= 0) w[i] = *reinterpret_cast<const uint4*>(x + src * ld + c0 + 8 * ch);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(s_x + tile_at(16 * i + rg, ch)) = w[i];
    if (ROWS) {
        // the rows' own codes: 16 threads hold one row's block
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 16 * i + rg;
            const B128Scale q = b128_scale(max16(absmax8(w[i])));
            if (r < nr) {
                if (8 * ch < nc)
                    *reinterpret_cast<uint2*>(codes + (first + r) * cols + c0 + 8 * ch) = b128_codes8(w[i], q.inv);
                if (ch == 0) scale[(int64_t)blockIdx.x * rows + first + r] = q.scale;
            }
        }
    }
    __syncthreads();
    // columns (the transposed codes go where the tile was once every thread
    // holds its share in registers): thread (p, q) takes channels 2p, 2p + 1 and rows 32q ..
    const int p = tid & 63, q = tid >> 6;
    uint32_t v[32], m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] = *reinterpret_cast<const uint32_t*>(s_x + tile_at(32 * q + i, p >> 2) + 4 * (p & 3));
        if (ROWS && tail) v[i] = 0;
        m = absmax2_bf16(m, v[i]);
    }
    s_max[q][2 * p] = m & 0xFFFFu;
    s_max[q][2 * p + 1] = m >> 16;
    __syncthreads();
    const B128Scale a = b128_scale(max(max(s_max[0][2 * p], s_max[1][2 * p]), max(s_max[2][2 * p], s_max[3][2 * p])));
    const B128Scale b = b128_scale(
        max(max(s_max[0][2 * p + 1], s_max[1][2 * p + 1]), max(s_max[2][2 * p + 1], s_max[3][2 * p + 1])));
    if (q == 0 && 2 * p < nc) {
        t_scale[blk * cols + c0 + 2 * p] = a.scale;
        t_scale[blk * cols + c0 + 2 * p + 1] = b.scale;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        *reinterpret_cast<uint32_t*>(s_x + TILE_T * (2 * p) + 32 * q + i) =
            e4m3x4(bf16_lo(v[i]) * a.inv, bf16_lo(v[i + 1]) * a.inv, bf16_lo(v[i + 2]) * a.inv, bf16_lo(v[i + 3]) * a.inv);
        *reinterpret_cast<uint32_t*>(s_x + TILE_T * (2 * p + 1) + 32 * q + i) =
            e4m3x4(bf16_hi(v[i]) * b.inv, bf16_hi(v[i + 1]) * b.inv, bf16_hi(v[i + 2]) * b.inv, bf16_hi(v[i + 3]) * b.inv);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = 32 * i + (tid >> 3), k = tid & 7;
        const uint32_t* s = reinterpret_cast<const uint32_t*>(s_x + TILE_T * c + 16 * k);
        if (c < nc)
            *reinterpret_cast<uint4*>(t_codes + (int64_t)(c0 + c) * P + 128 * blk + 16 * k) =
                make_uint4(s[0], s[1], s[2], s[3]);
    }
}

// Weights: one workgroup per 128 x 128 block of one expert.
template <bool TRANS>
__global__ __launch_bounds__(256) void k_quantize_b128_weights(const uint16_t* __restrict__ w, int n, int k,
                                                               int64_t ld, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ codes_t,
                                                               float* __restrict__ scale) {
    __shared__ __align__(16) uint8_t s_c[128 * TILE_T];  // codes of the block by row
    __shared__ uint32_t s_max[4];
    const int tid = threadIdx.x;
    const int64_t e = blockIdx.z;
    const int n0 = blockIdx.y * 128, k0 = blockIdx.x * 128;
    const int nr = min(128, n - n0), nc = min(128, k - k0);
    const int ch = tid & 15, rg = tid >> 4;
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 16 * i + rg;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < nr && 8 * ch < nc) v[i] = *reinterpret_cast<const uint4*>(w + (e * n + n0 + r) * ld + k0 + 8 * ch);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, absmax8(v[i]));
    m = wave_max_u32(m);
    if ((tid & 63) == 0) s_max[tid >> 6] = m;
    __syncthreads();
    const B128Scale q = b128_scale(max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3])));
    if (tid == 0) scale[(e * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = q.scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 16 * i + rg;
        const uint2 c = b128_codes8(v[i], q.inv);
        if (r < nr && 8 * ch < nc) *reinterpret_cast<uint2*>(codes + (e * n + n0 + r) * k + k0 + 8 * ch) = c;
        if (TRANS) {
            uint32_t* s = reinterpret_cast<uint32_t*>(s_c + TILE_T * r + 8 * ch);
            s[0] = c.x;
            s[1] = c.y;
        }
    }
    if constexpr (TRANS) {
        __syncthreads();
        // thread: 4 columns x 16 rows, four 4 x 4 byte transposes; 16 bytes of
        // each of 4 output rows, 8 neighbouring threads a whole 128-byte row
        const int rq = tid & 7, cg = tid >> 3;
        uint32_t o[4][4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[i] = *reinterpret_cast<const uint32_t*>(s_c + TILE_T * (16 * rq + 4 * b + i) + 4 * cg);
            const uint32_t a0 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), a1 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
            const uint32_t b0 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u), b1 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
            o[0][b] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
            o[1][b] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
            o[2][b] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
            o[3][b] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
        }
        if (16 * rq < nr) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * cg + j < nc)
                    *reinterpret_cast<uint4*>(codes_t + (e * k + k0 + 4 * cg + j) * (int64_t)n + n0 + 16 * rq) =
                        make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
        }
    }
}

namespace {
bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
}  // namespace
}  // namespace bsq

extern "C" {

bsq_status bsq_quantize_fp8b128(const void* x_bf16, int64_t src_rows, int64_t cols, int64_t ld_x,
                                const int32_t* row_index, int64_t rows, const int32_t* offsets, int32_t num_groups,
                                uint8_t* codes, float* scale, uint8_t* t_codes, float* t_scale, hipStream_t stream) {
    if (src_rows < 0 || cols < 0 || rows < 0 || num_groups < 0) return BSQ_ERR_INVALID_ARG;
    if ((codes == nullptr) != (scale == nullptr) || (t_codes == nullptr) != (t_scale == nullptr))
        return BSQ_ERR_INVALID_ARG;
    if (!codes && !t_codes) return BSQ_ERR_INVALID_ARG;
    if (!row_index && rows != src_rows) return BSQ_ERR_INVALID_ARG;
    if (t_codes && (!offsets || num_groups < 1)) return BSQ_ERR_INVALID_ARG;
    if (cols == 0 || (rows == 0 && !t_codes)) return BSQ_OK;
    if ((src_rows > 0 && rows > 0 && !x_bf16) || ld_x < cols) return BSQ_ERR_INVALID_ARG;
    if (cols % 16 || ld_x % 8 || !bsq::al(x_bf16, 16) || !bsq::al(codes, 16) || !bsq::al(t_codes, 16) ||
        !bsq::al(scale, 4) || !bsq::al(t_scale, 4) || !bsq::al(row_index, 4) || !bsq::al(offsets, 4))
        return BSQ_ERR_UNSUPPORTED;
    const int64_t P = bsq_colwise_padded_cols(num_groups, rows);
    if (cols > ((int64_t)1 << 22) || src_rows >= (int64_t)1 << 31 || rows > ((int64_t)1 << 27)) return BSQ_ERR_UNSUPPORTED;
    const uint16_t* x = static_cast<const uint16_t*>(x_bf16);
    if (t_codes && P / 128 > 65535) return BSQ_ERR_UNSUPPORTED;
    if (!t_codes) {
        const dim3 grid((unsigned)((rows + bsq::ROWS_R - 1) / bsq::ROWS_R),
                        (unsigned)((cols + 128 * bsq::ROWS_B - 1) / (128 * bsq::ROWS_B)));
        if (row_index)
            hipLaunchKernelGGL((bsq::k_quantize_b128_rows<true>), grid, dim3(256), 0, stream, x, rows, (int)cols, ld_x,
                               row_index, src_rows, codes, scale);
        else
            hipLaunchKernelGGL((bsq::k_quantize_b128_rows<false>), grid, dim3(256), 0, stream, x, rows, (int)cols,
                               ld_x, row_index, src_rows, codes, scale);
        return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
    }
    const dim3 grid((unsigned)((cols + 127) / 128), (unsigned)(P / 128));
#define BSQ_B128_COLS(GATHER, ROWS)                                                                                \
    hipLaunchKernelGGL((bsq::k_quantize_b128_cols<GATHER, ROWS>), grid, dim3(256), 0, stream, x, rows, (int)cols,  \
                       ld_x, row_index, src_rows, offsets, num_groups, P, codes, scale, t_codes, t_scale)
    if (codes) {
        if (row_index) BSQ_B128_COLS(true, true);
        else BSQ_B128_COLS(false, true);
    } else {
        if (row_index) BSQ_B128_COLS(true, false);
        else BSQ_B128_COLS(false, false);
    }
#undef BSQ_B128_COLS
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}

bsq_status bsq_quantize_fp8b128_weights(const void* w_bf16, int32_t num_experts, int64_t n, int64_t k, int64_t ld_w,
                                        uint8_t* codes, uint8_t* codes_t, float* scale, hipStream_t stream) {
    if (num_experts < 0 || n < 0 || k < 0) return BSQ_ERR_INVALID_ARG;
    if (num_experts == 0 || n == 0 || k == 0) return BSQ_OK;
    if (!w_bf16 || !codes || !scale || ld_w < k) return BSQ_ERR_INVALID_ARG;
    if (n % 16 || k % 16 || ld_w % 8 || !bsq::al(w_bf16, 16) || !bsq::al(codes, 16) || !bsq::al(codes_t, 16) ||
        !bsq::al(scale, 4))
        return BSQ_ERR_UNSUPPORTED;
    if (n > ((int64_t)1 << 22) || k > ((int64_t)1 << 22) || num_experts > 65535) return BSQ_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)((k + 127) / 128), (unsigned)((n + 127) / 128), (unsigned)num_experts);
    const uint16_t* w = static_cast<const uint16_t*>(w_bf16);
    if (codes_t)
        hipLaunchKernelGGL((bsq::k_quantize_b128_weights<true>), grid, dim3(256), 0, stream, w, (int)n, (int)k, ld_w,
                           codes, codes_t, scale);
    else
        hipLaunchKernelGGL((bsq::k_quantize_b128_weights<false>), grid, dim3(256), 0, stream, w, (int)n, (int)k, ld_w,
                           codes, codes_t, scale);
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}

}  // extern "C"
