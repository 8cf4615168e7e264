// Expert grouped GEMMs on E4M3 operands with one fp32 scale per 128 elements.
//
// All three products are "reduction-contiguous": C[r][c] = sum_b sA[b][r]
// sB[b][c] sum_{t in block b} A[r][t] B[c][t], blocks of 128 along t:
//   forward  A = activation rows of expert e, B = rows of W_e, t = k;
//            sB is one value per 128 x 128 weight block;
//   dgrad    A = rows of dY, B = rows of W_e^T, t = n; sB as above, transposed;
//   wgrad    A = rows of dY^T, B = rows of X^T, t = the expert's tokens;
//            sB is one value per row of B, like sA.
// The matrix core sums a block's 128 products (v_mfma_f32_16x16x128_f8f6f4, K =
// one block, a zero accumulator), and the vector units add the block into the
// fp32 accumulators with its scales: 4 FMAs per 16 x 16 x 128 MFMA forward, 4
// multiplies more for wgrad, which run beside the next MFMA (32 cycles).
//
// Operand order: B supplies the MFMA's rows and A its columns, so lane l holds
// output row l % 16 and the four adjacent output columns 4 (l / 16) ..+3 of
// each 16 x 16 tile: one row scale per lane, and stores of adjacent columns.
// Any order of t inside a block gives the same sum as long as both operands
// use it: lane l takes 16-byte chunks l / 16 and 4 + l / 16 of a 128-byte row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bsq.h"
#include "device_common.h"
#include "gemm_common.h"
#include "gemm_pipe.h"
#include "moe_common.h"

namespace bsq {

struct B128Args {
    const uint8_t* a;
    const float* as;
    const uint8_t* b;
    const float* bs;
    const int32_t* offsets;
    int E;
    int64_t M;       // rows of the token dimension
    int64_t R;       // forward / dgrad: reduction length; wgrad: rows of A per expert (n)
    int64_t C;       // output columns
    int64_t P;       // wgrad: pitch of the token-column codes
    int64_t bs_e, bs_c, bs_b;  // strides of sB by expert, 128-column block and reduction block
    void* out;
    int32_t* err;    // error word
};

// ds_read_b128 fragment of 16 rows x 128 bytes at `base` (rows of 128 bytes,
// chunk c of row r at slot c ^ swz8(r)).
__device__ __forceinline__ int8v b128_frag(const __attribute__((address_space(3))) uint8_t* lds, uint32_t base, int lane) {
    const int r = lane & 15, g = lane >> 4;
    const uint32_t at = base + 128u * (uint32_t)r + 16u * (uint32_t)(g ^ swz8(r));
    const u32x4 x0 = *(const __attribute__((address_space(3))) u32x4*)(lds + at);
    const u32x4 x1 = *(const __attribute__((address_space(3))) u32x4*)(lds + (at ^ 64u));
    return int8v{(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
}

__device__ __forceinline__ float4v b128_mfma(const int8v& b, const int8v& a) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, float4v{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// Where row tile `rt` (of TM rows) lies: expert e (E for the rows past the last
// one) and its row range; e = -1 past the end or where the offsets are
// invalid.  Every wave scans the expert sizes 64 at a time.
struct RowTile {
    int e;
    int64_t row0, end;
};
template <int TM>
__device__ __forceinline__ RowTile find_row_tile(const B128Args& p, int64_t rt, int lane) {
    RowTile f{-1, 0, 0};
    int64_t before = 0;
    bool bad = p.offsets[0] != 0;
    for (int base = 0; base <= p.E; base += 64) {
        const int e = base + lane;
        int64_t lo = 0, hi = 0;
        if (e <= p.E) {
            lo = p.offsets[e];
            hi = e < p.E ? (int64_t)p.offsets[e + 1] : p.M;
        }
        bad |= __ballot(hi < lo) != 0;
        const int n = hi > lo ? (int)((hi - lo + TM - 1) / TM) : 0;
        const int incl = wave_scan_i32(n);
        const int64_t at = rt - before;
        const uint64_t in = __ballot(at >= incl - n && at < incl);
        if (in) {
            const int w = __builtin_ctzll(in);
            f.e = __builtin_amdgcn_readlane(e, w);
            const int lo_w = __builtin_amdgcn_readlane((int)lo, w), first = __builtin_amdgcn_readlane(incl - n, w);
            f.end = __builtin_amdgcn_readlane((int)hi, w);
            f.row0 = lo_w + (at - first) * TM;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    if (bad) f.e = -1;
    if (rt == 0 && lane == 0) *p.err = bad ? 1 : 0;
    return f;
}

// 128 x 128 output tiles: 4 waves of 64 x 64, a ring of two 128-byte stages
// per operand filled by buffer-to-LDS DMA, two workgroups per CU.
constexpr int BT = 128;
struct B128Slot {
    uint8_t a[BT * 128];
    uint8_t b[BT * 128];
    float sa[BT];
    float sb[BT];
};

template <bool OUT_F32, bool WGRAD>
__global__ __launch_bounds__(256, 2) void k_gemm_b128_tile(B128Args p) {
    __shared__ __align__(16) B128Slot s_ring[2];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int CT = (int)((p.C + BT - 1) / BT);
    int e, rows;
    int64_t r0, R;
    const uint8_t *a, *b;
    const float *as, *bs;
    int64_t lda, ldas, ldbs;
    char* out;
    int c0;
    if constexpr (!WGRAD) {
        // groups of 8 row tiles sweep the column tiles together
        const int64_t t = blockIdx.x;
        const int64_t g = t / (8 * CT);
        const int l = (int)(t - g * 8 * CT);
        const RowTile f = find_row_tile<BT>(p, g * 8 + (l & 7), lane);
        if (f.e < 0) return;
        e = f.e;
        r0 = f.row0;
        rows = (int)min((int64_t)BT, f.end - r0);
        c0 = BT * (l >> 3);
        R = e < p.E ? p.R : 0;
        const int64_t we = e < p.E ? e : 0;
        a = p.a + r0 * p.R;
        lda = p.R;
        as = p.as + r0;
        ldas = p.M;
        b = p.b + (we * p.C + c0) * p.R;
        bs = p.bs + we * p.bs_e + (int64_t)(c0 / BT) * p.bs_c;
        ldbs = p.bs_b;
        out = static_cast<char*>(p.out) + (r0 * p.C + c0) * (OUT_F32 ? 4 : 2);
    } else {
        const int RT = (int)((p.R + BT - 1) / BT);
        const int64_t t = blockIdx.x;
        e = (int)(t / (RT * CT));
        const int l = (int)(t - (int64_t)e * RT * CT);
        r0 = BT * (l % RT);
        c0 = BT * (l / RT);
        rows = (int)min((int64_t)BT, p.R - r0);
        // the whole call is dropped where any offset is invalid
        bool bad = p.offsets[0] != 0 || p.offsets[p.E] > p.M;
        for (int i = lane; i < p.E; i += 64) bad |= p.offsets[i + 1] < p.offsets[i];
        bad = __ballot(bad) != 0;
        if (t == 0 && threadIdx.x == 0) *p.err = bad ? 1 : 0;
        if (bad) return;
        const int64_t o0 = p.offsets[e];
        R = p.offsets[e + 1] - o0;
        const int64_t blk = e + o0 / 128;
        a = p.a + r0 * p.P + 128 * blk;
        lda = p.P;
        as = p.as + blk * p.R + r0;
        ldas = p.R;
        b = p.b + (int64_t)c0 * p.P + 128 * blk;
        bs = p.bs + blk * p.C + c0;
        ldbs = p.C;
        out = static_cast<char*>(p.out) + (((int64_t)e * p.R + r0) * p.C + c0) * (OUT_F32 ? 4 : 2);
    }
    const int cols = (int)min((int64_t)BT, p.C - c0);
    const int nb = (int)((R + 127) / 128);
    const uint32_t ld = __builtin_amdgcn_readfirstlane((uint32_t)lda);
    // token columns are padded to whole blocks of zeros; k and n are not
    const uint32_t len = WGRAD ? (uint32_t)nb * 128u : (uint32_t)R;
    const __amdgpu_buffer_rsrc_t ra = rsrc_n(uniform_ptr(a), 0x7FFFFFFFu), rb = rsrc_n(uniform_ptr(b), 0x7FFFFFFFu);
    const __amdgpu_buffer_rsrc_t rsa = rsrc_n(uniform_ptr(as), 0x7FFFFFFFu), rsb = rsrc_n(uniform_ptr(bs), 0x7FFFFFFFu);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(&s_ring[0]));
    const __attribute__((address_space(3))) uint8_t* lds =
        (const __attribute__((address_space(3))) uint8_t*)(&s_ring[0]);

    // Stage s into slot s & 1; 9 DMA instructions per wave.
    auto issue = [&](int s) {
        const uint32_t slot = lds0 + (uint32_t)(s & 1) * (uint32_t)sizeof(B128Slot);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 32 * wave + 8 * i + (lane >> 3);
            const uint32_t ko = 128u * (uint32_t)s + 16u * (uint32_t)((lane & 7) ^ swz8(row));
            const uint32_t dst = slot + 1024u * (uint32_t)(4 * wave + i);
            dma_lds_r<16>(ra, (row < rows && ko < len) ? (uint32_t)row * ld + ko : OOB, dst + (uint32_t)offsetof(B128Slot, a));
            dma_lds_r<16>(rb, (row < cols && ko < len) ? (uint32_t)row * ld + ko : OOB, dst + (uint32_t)offsetof(B128Slot, b));
        }
        const int h = wave & 1, row = 64 * h + lane;
        if (WGRAD && wave >= 2)
            dma_lds_r<4>(rsb, row < cols ? 4u * ((uint32_t)s * (uint32_t)ldbs + (uint32_t)row) : OOB,
                         slot + (uint32_t)offsetof(B128Slot, sb) + 256u * (uint32_t)h);
        else
            dma_lds_r<4>(rsa, row < rows ? 4u * ((uint32_t)s * (uint32_t)ldas + (uint32_t)row) : OOB,
                         slot + (uint32_t)offsetof(B128Slot, sa) + 256u * (uint32_t)h);
    };

    float4v acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};

    if (nb > 0) issue(0);
    for (int s = 0; s < nb; ++s) {
        if (s + 1 < nb) {
            issue(s + 1);
            wait_vmcnt<9>();
        } else {
            wait_vmcnt<0>();
        }
        block_barrier();
        const uint32_t slot = (uint32_t)(s & 1) * (uint32_t)sizeof(B128Slot);
        const float sw = WGRAD ? 1.0f : bs[s * ldbs];
        int8v fb[4];
        float4v sb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t c = (uint32_t)(64 * wn + 16 * j);
            fb[j] = b128_frag(lds, slot + (uint32_t)offsetof(B128Slot, b) + 128u * c, lane);
            if constexpr (WGRAD)
                sb[j] = *(const __attribute__((address_space(3))) float4v*)(
                    lds + slot + (uint32_t)offsetof(B128Slot, sb) + 4u * (c + 4u * (uint32_t)(lane >> 4)));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = (uint32_t)(64 * wm + 16 * i);
            const int8v fa = b128_frag(lds, slot + (uint32_t)offsetof(B128Slot, a) + 128u * r, lane);
            const float sa = *(const __attribute__((address_space(3))) float*)(
                lds + slot + (uint32_t)offsetof(B128Slot, sa) + 4u * (r + (uint32_t)(lane & 15)));
            const float sc = WGRAD ? sa : sa * sw;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4v d = b128_mfma(fb[j], fa);
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    acc[i][j][v] = fmaf(WGRAD ? d[v] * sb[j][v] : d[v], sc, acc[i][j][v]);
            }
        }
        wait_lgkmcnt0();
        block_barrier();
    }

    const __amdgpu_buffer_rsrc_t ro = make_rsrc(uniform_ptr(out), 0x7FFFFFFFu);
    const uint32_t ldo = (uint32_t)p.C * (OUT_F32 ? 4u : 2u);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 64 * wm + 16 * i + (lane & 15), c = 64 * wn + 16 * j + 4 * (lane >> 4);
            const bool ok = r < rows && c < cols;
            const uint32_t o = ok ? (uint32_t)r * ldo + (uint32_t)c * (OUT_F32 ? 4u : 2u) : OOB;
            if constexpr (OUT_F32)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), ro, (int)o, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b64(
                    u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])}, ro, (int)o,
                    0, 0);
        }
}

namespace {

constexpr int64_t kMaxOffset = (int64_t)1 << 31;  // 32-bit buffer offsets

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Most row tiles of TM rows that E experts and the rows past them can need.
int64_t max_row_tiles(int64_t M, int E, int TM) { return M / TM + (M < E + 1 ? M : E + 1); }

template <bool WGRAD>
bsq_status launch_b128(const B128Args& a, bool f32, hipStream_t s) {
    const int64_t ct = (a.C + BT - 1) / BT;
    int64_t grid;
    if (WGRAD)
        grid = (int64_t)a.E * ((a.R + BT - 1) / BT) * ct;
    else
        grid = (max_row_tiles(a.M, a.E, BT) + 7) / 8 * 8 * ct;
    if (grid * 256 >= (int64_t)1 << 32) return BSQ_ERR_UNSUPPORTED;
    if (f32)
        hipLaunchKernelGGL((k_gemm_b128_tile<true, WGRAD>), dim3((unsigned)grid), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_gemm_b128_tile<false, WGRAD>), dim3((unsigned)grid), dim3(256), 0, s, a);
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}

}  // namespace
}  // namespace bsq

extern "C" {

size_t bsq_grouped_gemm_fp8b128_workspace_size(int32_t num_experts) {
    if (num_experts < 1 || num_experts > bsq::MAX_EXPERTS) return 0;
    return 2 * (size_t)((bsq::plan_words(num_experts + 1) * 4 + 255) / 256 * 256);
}

bsq_status bsq_grouped_gemm_fp8b128_fwd(const uint8_t* a_codes, const float* a_scale, const uint8_t* w_codes,
                                        const float* w_scale, const int32_t* offsets, int32_t num_experts,
                                        int64_t m_total, int64_t n, int64_t k, void* y, bsq_dtype y_dtype,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (num_experts < 1 || m_total < 0 || n < 0 || k < 0) return BSQ_ERR_INVALID_ARG;
    if (y_dtype != BSQ_BF16 && y_dtype != BSQ_F32) return BSQ_ERR_INVALID_ARG;
    if (!offsets || !workspace || !w_codes || !w_scale) return BSQ_ERR_INVALID_ARG;
    if (m_total > 0 && (!a_codes || !a_scale || !y)) return BSQ_ERR_INVALID_ARG;
    if (num_experts > bsq::MAX_EXPERTS || n == 0 || k == 0 || n % 16 || k % 16) return BSQ_ERR_UNSUPPORTED;
    if (!bsq::al(a_codes, 16) || !bsq::al(w_codes, 16) || !bsq::al(a_scale, 4) || !bsq::al(w_scale, 4) ||
        !bsq::al(offsets, 4) || !bsq::al(y, 16) || !bsq::al(workspace, 256))
        return BSQ_ERR_UNSUPPORTED;
    // per-tile offsets are 32-bit: 256 rows of codes and outputs, the scales of all rows
    if (256 * k >= bsq::kMaxOffset || 256 * n * 4 >= bsq::kMaxOffset || m_total >= (int64_t)1 << 31 ||
        (k / 128 + 2) * m_total * 4 >= bsq::kMaxOffset)
        return BSQ_ERR_UNSUPPORTED;
    if (workspace_bytes < bsq_grouped_gemm_fp8b128_workspace_size(num_experts)) return BSQ_ERR_WORKSPACE_TOO_SMALL;
    if (m_total == 0) return BSQ_OK;
    const int64_t kb = (k + 127) / 128, nb = (n + 127) / 128;
    const bsq::B128Args a{a_codes, a_scale, w_codes, w_scale, offsets, num_experts, m_total, k, n, 0,
                          nb * kb, kb, 1, y, static_cast<int32_t*>(workspace) + bsq::PLAN_ERR};
    return bsq::launch_b128<false>(a, y_dtype == BSQ_F32, stream);
}

bsq_status bsq_grouped_gemm_fp8b128_bwd(const uint8_t* dy_codes, const float* dy_scale, const uint8_t* wt_codes,
                                        const float* w_scale, const uint8_t* dyt_codes, const float* dyt_scale,
                                        const uint8_t* xt_codes, const float* xt_scale, const int32_t* offsets,
                                        int32_t num_experts, int64_t m_total, int64_t n, int64_t k, void* dx,
                                        bsq_dtype dx_dtype, void* dw, bsq_dtype dw_dtype, unsigned flags,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (num_experts < 1 || m_total < 0 || n < 0 || k < 0) return BSQ_ERR_INVALID_ARG;
    if (flags == 0 || (flags & ~(BSQ_DGRAD | BSQ_WGRAD)) || !offsets || !workspace) return BSQ_ERR_INVALID_ARG;
    const bool dg = flags & BSQ_DGRAD, wg = flags & BSQ_WGRAD;
    if (dg && dx_dtype != BSQ_BF16 && dx_dtype != BSQ_F32) return BSQ_ERR_INVALID_ARG;
    if (wg && dw_dtype != BSQ_BF16 && dw_dtype != BSQ_F32) return BSQ_ERR_INVALID_ARG;
    if (dg && (!wt_codes || !w_scale || (m_total > 0 && (!dy_codes || !dy_scale || !dx)))) return BSQ_ERR_INVALID_ARG;
    if (wg && (!dyt_codes || !dyt_scale || !xt_codes || !xt_scale || !dw)) return BSQ_ERR_INVALID_ARG;
    if (num_experts > bsq::MAX_EXPERTS || n == 0 || k == 0 || n % 16 || k % 16) return BSQ_ERR_UNSUPPORTED;
    if (!bsq::al(offsets, 4) || !bsq::al(workspace, 256)) return BSQ_ERR_UNSUPPORTED;
    if (dg && (!bsq::al(dy_codes, 16) || !bsq::al(dy_scale, 4) || !bsq::al(wt_codes, 16) || !bsq::al(w_scale, 4) ||
               !bsq::al(dx, 16)))
        return BSQ_ERR_UNSUPPORTED;
    if (wg && (!bsq::al(dyt_codes, 16) || !bsq::al(dyt_scale, 4) || !bsq::al(xt_codes, 16) || !bsq::al(xt_scale, 4) ||
               !bsq::al(dw, 16)))
        return BSQ_ERR_UNSUPPORTED;
    const int64_t P = bsq_colwise_padded_cols(num_experts, m_total);
    if (m_total >= (int64_t)1 << 31 || 256 * k * 4 >= bsq::kMaxOffset ||
        (dg && (256 * n >= bsq::kMaxOffset || (n / 128 + 2) * m_total * 4 >= bsq::kMaxOffset)) ||
        (wg && (256 * P >= bsq::kMaxOffset || P / 128 * (n > k ? n : k) * 4 >= bsq::kMaxOffset)))
        return BSQ_ERR_UNSUPPORTED;
    if (workspace_bytes < bsq_grouped_gemm_fp8b128_workspace_size(num_experts)) return BSQ_ERR_WORKSPACE_TOO_SMALL;
    const int64_t kb = (k + 127) / 128, nb = (n + 127) / 128;
    int32_t* err = static_cast<int32_t*>(workspace) + bsq::PLAN_ERR;
    if (dg && m_total > 0) {
        const bsq::B128Args a{dy_codes, dy_scale, wt_codes, w_scale, offsets, num_experts, m_total, n, k, 0,
                              nb * kb, 1, kb, dx, err};
        const bsq_status st = bsq::launch_b128<false>(a, dx_dtype == BSQ_F32, stream);
        if (st != BSQ_OK) return st;
    }
    if (wg) {
        const bsq::B128Args a{dyt_codes, dyt_scale, xt_codes, xt_scale, offsets, num_experts, m_total, n, k, P,
                              0, 0, 0, dw, err};
        return bsq::launch_b128<true>(a, dw_dtype == BSQ_F32, stream);
    }
    return BSQ_OK;
}

}  // extern "C"
