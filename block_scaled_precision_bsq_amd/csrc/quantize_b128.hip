// E4M3 codes with one fp32 scale per 128 elements: rows of activations
// (1 x 128 along a row, the rows optionally gathered), token columns of each
// expert (128 x 1 down its rows, transposed output) and weights (128 x 128,
// both orientations).
//
// A block with maximum magnitude a: c = max(a, 2^-100), code of x =
// E4M3_RNE(RN(x * RN(448 / c))) (saturating: the product may round past 448),
// scale = RN(c / 448), and 0 for an all-zero block; a block that holds an
// infinity or a NaN gets a NaN scale (as magnitude bits those order above all
// finite numbers), so no element of it passes for a number.  The two divisions are
// correctly rounded, once per block; an element costs an unpack, a multiply and
// its share of a packed conversion.  The product is below 448 (1 + 2^-23), which
// rounds to 448, so there is no clamp.  With few enough instructions around
// them every kernel here is bound by its bytes: 2 per element read, 1 or 2
// written.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsq.h"
#include "device_common.h"

namespace bsq {

constexpr float B128_TINY = 0x1p-100f;
// Cache policy of the code stores: non-temporal.  They are whole 128-byte lines
// that the kernel does not read (with ordinary stores 137 us instead of 117 for
// 4096 tokens gathered into 32768 x 7168 row and column codes: 0.52 GB written,
// 0.27 GB fetched past L2).
constexpr int NT = 2;

struct B128Scale {
    float inv, scale;
};
// From the maximum's bf16 magnitude bits.  A quotient estimate q with its exact
// remainder r gives RN(q + r y) with y the reciprocal: before the rounding it is
// within 2^-45 of the true quotient, and a quotient of integers below 2^8
// (448 = 7 * 64; c has 8 bits) is either a binary32 number or at least 2^-33 away
// from the middle of two.
__device__ __forceinline__ B128Scale b128_scale(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits << 16);
    // (no maximum: a NaN has to stay; an infinite c gives 0 * inf below)
    const float c = a < B128_TINY ? B128_TINY : a;
    // (c moved towards 1, where its reciprocal is a normal number)
    const float f = c > 1.0f ? 0x1p-60f : 0x1p60f, d = c * f;
    const float y = __builtin_amdgcn_rcpf(d), z = 1.0f / 448.0f;
    const float q = 448.0f * y, p = c * z;
    const float inv = fmaf(fmaf(-d, q, 448.0f), y, q) * f;
    const float scale = fmaf(fmaf(-448.0f, p, c), z, p);
    return {inv, a == 0.0f ? 0.0f : scale};
}

// E4M3 bytes of four floats of magnitude below 464, a in the lowest byte.
__device__ __forceinline__ uint32_t b128_e4m3x4(float a, float b, float c, float d) {
    return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}

// E4M3 codes of four packed pairs (8 elements) times inv.
__device__ __forceinline__ uint2 b128_codes8(uint4 w, float inv) {
    return make_uint2(b128_e4m3x4(bf16_lo(w.x) * inv, bf16_hi(w.x) * inv, bf16_lo(w.y) * inv, bf16_hi(w.y) * inv),
                      b128_e4m3x4(bf16_lo(w.z) * inv, bf16_hi(w.z) * inv, bf16_lo(w.w) * inv, bf16_hi(w.w) * inv));
}

__device__ __forceinline__ uint32_t absmax8(uint4 w) {
    return fold_max16(absmax2_bf16(absmax2_bf16(absmax2_bf16(w.x & 0x7FFF7FFFu, w.y), w.z), w.w));
}

// Lane moves within rows of 16.
template <int CTRL>
__device__ __forceinline__ uint32_t row_move(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}

// Eight maxima over the 16 lanes of a row, scattered: lane l gets the one of
// m[l / 2].  Each step halves the values a lane works on: it keeps those of its
// half and takes the partner's share of them, partners l ^ 8, l ^ 7, l ^ 2, and
// last adds l ^ 1.
__device__ __forceinline__ uint32_t scatter_max16(const uint32_t (&m)[8], int l) {
    uint32_t a[4], b[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = max((l & 8) ? m[i + 4] : m[i], row_move<0x128>((l & 8) ? m[i] : m[i + 4]));
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = max((l & 4) ? a[i + 2] : a[i], row_move<0x141>((l & 4) ? a[i] : a[i + 2]));
    const uint32_t c = max((l & 2) ? b[1] : b[0], row_move<0x4E>((l & 2) ? b[0] : b[1]));
    return max(c, row_move<0xB1>(c));
}
// The value that lane 2 I of the row holds.
template <int I>
__device__ __forceinline__ float row_value(float x) { return __uint_as_float(row_move<0x150 + 2 * I>(__float_as_uint(x))); }

// Codes of eight pieces of 8 elements, the inverse of piece i in lane 2 i of
// the row; store(i, codes) takes them.
template <class F>
__device__ __forceinline__ void codes_of_row(const uint4 (&w)[8], float inv, F store) {
    store(0, b128_codes8(w[0], row_value<0>(inv)));
    store(1, b128_codes8(w[1], row_value<1>(inv)));
    store(2, b128_codes8(w[2], row_value<2>(inv)));
    store(3, b128_codes8(w[3], row_value<3>(inv)));
    store(4, b128_codes8(w[4], row_value<4>(inv)));
    store(5, b128_codes8(w[5], row_value<5>(inv)));
    store(6, b128_codes8(w[6], row_value<6>(inv)));
    store(7, b128_codes8(w[7], row_value<7>(inv)));
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
    uint32_t m[ROWS_B];
#pragma unroll
    for (int b = 0; b < ROWS_B; ++b) m[b] = absmax8(w[b]);
    const B128Scale q = b128_scale(scatter_max16(m, l));
    if ((l & 1) == 0) s_scale[l >> 1][g] = q.scale;
    codes_of_row(w, q.inv, [&](int b, uint2 v) {
        const int c = 128 * (b0 + b) + 8 * l;
        if (r < rows && c < cols) *reinterpret_cast<uint2*>(codes + r * cols + c) = v;
    });
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
    __shared__ uint32_t s_max[4][64];  // two 16-bit magnitudes
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
    const int64_t first = uniform_i64(o0 + 128 * (blk - grp - max((int64_t)0, o0) / 128));
    const int nr = __builtin_amdgcn_readfirstlane(
        (o0 >= 0 && first >= o0) ? (int)max((int64_t)0, min((int64_t)128, o1 - first)) : 0);

    // load: 16 threads a row, 8 steps of 16 rows
    const bool need = ROWS || !tail;
    const int ch = tid & 15, rg = tid >> 4;
    uint4 w[8];
    if constexpr (GATHER) {
        const uint16_t* xc = x + c0 + 8 * ch;
        const int limit = (need && 8 * ch < nc) ? nr : 0;
        int32_t src[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) src[i] = 16 * i + rg < limit ? row_index[first + 16 * i + rg] : -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = make_uint4(0, 0, 0, 0);
            if ((uint32_t)src[i] < (uint32_t)src_rows)
                w[i] = *reinterpret_cast<const uint4*>(xc + (uint64_t)(uint32_t)src[i] * (uint32_t)ld);
        }
    } else {
        // rows past the tile lie past the resource's range
        const __amdgpu_buffer_rsrc_t rx =
            make_rsrc(uniform_ptr(x + first * ld + c0), (need && nr > 0) ? 2u * ((uint32_t)(nr - 1) * (uint32_t)ld + (uint32_t)nc) : 0u);
        const uint32_t o = 8 * ch < nc ? 2u * ((uint32_t)rg * (uint32_t)ld + 8u * (uint32_t)ch) : OOB;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = buf_load16(rx, o + (uint32_t)(32 * i) * (uint32_t)ld);
    }
    const uint32_t put = tile_at(rg, ch);
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(s_x + put + 4096u * i) = w[i];
    if (ROWS) {
        // the rows' own codes: 16 threads hold one row's block
        uint32_t m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = absmax8(w[i]);
        const B128Scale q = b128_scale(scatter_max16(m, ch));
        const int mine = 16 * (ch >> 1) + rg;  // the row whose scale this lane has
        if ((ch & 1) == 0 && mine < nr) scale[(int64_t)blockIdx.x * rows + first + mine] = q.scale;
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(uniform_ptr(codes + first * cols + c0),
                                                    nr > 0 ? (uint32_t)(nr - 1) * (uint32_t)cols + (uint32_t)nc : 0u);
        const uint32_t o = 8 * ch < nc ? (uint32_t)rg * (uint32_t)cols + 8u * (uint32_t)ch : OOB;
        codes_of_row(w, q.inv, [&](int i, uint2 v) {
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{v.x, v.y}, rc, (int)(o + (uint32_t)(16 * i) * (uint32_t)cols), 0, NT);
        });
    }
    // columns past the tile lie past the resource's range
    const __amdgpu_buffer_rsrc_t rt = make_rsrc(uniform_ptr(t_codes + (int64_t)c0 * P + 128 * blk), (uint32_t)(nc - 1) * (uint32_t)P + 128u);
    const uint32_t to = (uint32_t)(tid >> 3) * (uint32_t)P + 16u * (uint32_t)(tid & 7);
    if (tail || nr == 0) {
        const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) __builtin_amdgcn_raw_buffer_store_b128(zero, rt, (int)(to + (uint32_t)(32 * i) * (uint32_t)P), 0, NT);
        if (tid < nc) t_scale[blk * cols + c0 + tid] = 0.0f;
        return;
    }
    __syncthreads();
    // columns (the transposed codes go where the tile was once every thread
    // holds its share in registers): thread (p, q) takes channels 2p, 2p + 1 and rows 32q ..
    const int p = tid & 63, q = tid >> 6;
    uint32_t v[32], m = 0;
    const uint32_t get = (uint32_t)(8192 * q + 16 * (p >> 2) + 4 * (p & 3));  // tile_at(32 q, p / 4)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t at = get ^ (uint32_t)(16 * i);
        v[i] = *reinterpret_cast<const uint32_t*>(s_x + at + 256 * i);
        v[i + 16] = *reinterpret_cast<const uint32_t*>(s_x + at + 256 * (i + 16));
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) m = absmax2_bf16(m, v[i]);
    *reinterpret_cast<uint32_t*>(&s_max[q][p]) = m;
    __syncthreads();
    m = absmax2_bf16(absmax2_bf16(s_max[0][p], s_max[1][p]), absmax2_bf16(s_max[2][p], s_max[3][p]));
    const B128Scale a = b128_scale(m & 0xFFFFu), b = b128_scale(m >> 16);
    if (q == 0 && 2 * p < nc) {
        t_scale[blk * cols + c0 + 2 * p] = a.scale;
        t_scale[blk * cols + c0 + 2 * p + 1] = b.scale;
    }
    uint32_t* ta = reinterpret_cast<uint32_t*>(s_x + TILE_T * (2 * p) + 32 * q);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        ta[i / 4] = b128_e4m3x4(bf16_lo(v[i]) * a.inv, bf16_lo(v[i + 1]) * a.inv, bf16_lo(v[i + 2]) * a.inv, bf16_lo(v[i + 3]) * a.inv);
        ta[TILE_T / 4 + i / 4] =
            b128_e4m3x4(bf16_hi(v[i]) * b.inv, bf16_hi(v[i + 1]) * b.inv, bf16_hi(v[i + 2]) * b.inv, bf16_hi(v[i + 3]) * b.inv);
    }
    __syncthreads();
    const uint32_t* ts = reinterpret_cast<const uint32_t*>(s_x + TILE_T * (tid >> 3) + 16 * (tid & 7));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t* c = ts + 32 * i * (TILE_T / 4);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4{c[0], c[1], c[2], c[3]}, rt, (int)(to + (uint32_t)(32 * i) * (uint32_t)P), 0, NT);
    }
}

// Weights: one workgroup per 128 x 128 block of one expert.  32 x 4096 x 7168:
// 706 us, 5.3 TB/s, where a device copy of 2 GiB moves 4.9 to 5.1 (another card 674,
// and there 696 with ordinary loads and stores).
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
        if (r < nr && 8 * ch < nc) v[i] = ld_stream16(w + (e * n + n0 + r) * ld + k0 + 8 * ch);
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
        if (r < nr && 8 * ch < nc) st_stream8(codes + (e * n + n0 + r) * k + k0 + 8 * ch, c);
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
                    st_stream16(codes_t + (e * k + k0 + 4 * cg + j) * (int64_t)n + n0 + 16 * rq,
                                make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]));
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
    if (cols == 0) return BSQ_OK;
    // (without rows the row form has no bytes, and an index no address)
    if (rows > 0 && ((!codes && !t_codes) || (!row_index && rows != src_rows))) return BSQ_ERR_INVALID_ARG;
    if (t_codes && (!offsets || num_groups < 1)) return BSQ_ERR_INVALID_ARG;
    if (rows == 0 && !t_codes) return BSQ_OK;
    if ((src_rows > 0 && rows > 0 && !x_bf16) || ld_x < cols) return BSQ_ERR_INVALID_ARG;
    if (cols % 16 || ld_x % 8 || !bsq::al(x_bf16, 16) || !bsq::al(codes, 16) || !bsq::al(t_codes, 16) ||
        !bsq::al(scale, 4) || !bsq::al(t_scale, 4) || !bsq::al(row_index, 4) || !bsq::al(offsets, 4))
        return BSQ_ERR_UNSUPPORTED;
    const int64_t P = bsq_colwise_padded_cols(num_groups, rows);
    if (cols > ((int64_t)1 << 22) || src_rows >= (int64_t)1 << 31 || rows > ((int64_t)1 << 27)) return BSQ_ERR_UNSUPPORTED;
    const uint16_t* x = static_cast<const uint16_t*>(x_bf16);
    if (t_codes && (P / 128 > 65535 || ld_x >= (int64_t)1 << 23)) return BSQ_ERR_UNSUPPORTED;  // 32-bit offsets in a tile
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
