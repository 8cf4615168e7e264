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
//
// Every tile size adds the blocks one after the other, by the same operations: what
// a row gets (wgrad: an expert) is the same bits whatever else the call holds.  No
// reduction is split, so few tiles with a long one get smaller tiles instead.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

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
    int even;        // tiles spread evenly over the XCDs (k_gemm_b128_tile)
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
// pick(all) names the row tile, from the number of all of them where ALL and p.even.
template <int TM, bool ALL, class Pick>
__device__ __forceinline__ RowTile pick_row_tile(const B128Args& p, int lane, Pick pick) {
    bool bad = p.offsets[0] != 0;
    int64_t lo, hi;
    int n, incl;
    auto sizes = [&](int base) {  // of the experts base + lane, their tiles and running count
        const int e = base + lane;
        lo = hi = 0;
        if (e <= p.E) {
            lo = p.offsets[e];
            hi = e < p.E ? (int64_t)p.offsets[e + 1] : p.M;
        }
        bad |= __ballot(hi < lo) != 0;
        n = hi > lo ? (int)((hi - lo + TM - 1) / TM) : 0;
        incl = wave_scan_i32(n);
    };
    sizes(0);
    int64_t all = __builtin_amdgcn_readlane(incl, 63);
    if (ALL && p.even && p.E >= 64) {
        for (int base = 64; base <= p.E; base += 64) {
            sizes(base);
            all += __builtin_amdgcn_readlane(incl, 63);
        }
        sizes(0);
    }
    const int64_t rt = pick(all);
    RowTile f{-1, 0, 0};
    int64_t before = 0;
    for (int base = 0;;) {
        const int64_t at = rt - before;
        const uint64_t in = __ballot(at >= incl - n && at < incl);
        if (in) {
            const int w = __builtin_ctzll(in);
            f.e = base + w;
            const int lo_w = __builtin_amdgcn_readlane((int)lo, w), first = __builtin_amdgcn_readlane(incl - n, w);
            f.end = __builtin_amdgcn_readlane((int)hi, w);
            f.row0 = lo_w + (at - first) * TM;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
        base += 64;
        if (base > p.E) break;
        sizes(base);
    }
    if (bad) f.e = -1;
    if (rt == 0 && lane == 0) *p.err = bad ? 1 : 0;
    return f;
}
template <int TM>
__device__ __forceinline__ RowTile find_row_tile(const B128Args& p, int64_t rt, int lane) {
    return pick_row_tile<TM, false>(p, lane, [&](int64_t) { return rt; });
}

// BT x BT output tiles, BT 32, 64 or 128: 4 waves of BT/2 x BT/2, a ring of two
// 128-byte stages per operand filled by buffer-to-LDS DMA, two workgroups or more per
// CU.  A stage's products take a fraction of its loads' latency, so two stages are in
// flight: 3001 rows over 12 experts of 1424 x 2000 28.9 us with BT 128 (with one 30.3;
// 12 us are the host's), 1024 rows over 32 experts of 4096 x 7168 197 us (273); three or
// four of them with BT 64 change nothing.  Where rows are few the weights' bytes bound
// it: 64 rows over 32 experts of 4096 x 7168 120 us with BT 64, 6.4 TB/s.
template <int BT>
struct B128Slot {
    uint8_t a[BT * 128];
    uint8_t b[BT * 128];
    float sa[BT < 64 ? 64 : BT];  // (a DMA instruction writes 64 lanes' words)
    float sb[BT < 64 ? 64 : BT];
};

template <bool OUT_F32, bool WGRAD, int BT, int B_AUX>
__global__ __launch_bounds__(256, 2) void k_gemm_b128_tile(B128Args p) {
    constexpr int NG = BT / 32;        // groups of 16 rows, and of 16 columns, of a wave
    constexpr int DMAS = 2 * NG + 1;   // DMA instructions per wave and stage
    typedef B128Slot<BT> Slot;
    __shared__ __align__(16) Slot s_ring[2];
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
    uint32_t tile = blockIdx.x;  // (grids stay below 2^24 workgroups)
    if constexpr (!WGRAD) {
        // An XCD gets every eighth workgroup.  Either eight row tiles sweep the column
        // tiles together, each on its XCD, or (p.even) an XCD takes an eighth of them,
        // row by row: as many as the others do (17 row tiles of 11 column tiles 36 us
        // against 55 the other way, where one XCD gets three of them and another two;
        // many rounds of 128 x 128 tiles up to 5% slower).
        bool on = true;
        const RowTile f = pick_row_tile<BT, true>(p, lane, [&](int64_t all) {
            if (p.even) {
                const uint32_t n = (uint32_t)all * (uint32_t)CT, share = (n + 7) / 8, i = blockIdx.x >> 3;
                tile = (blockIdx.x & 7) * share + i;
                on = i < share && tile < n;
            } else {
                const uint32_t g = tile / (8u * (uint32_t)CT), l = tile - g * 8u * (uint32_t)CT;
                tile = (g * 8 + (l & 7)) * (uint32_t)CT + (l >> 3);
            }
            return (int64_t)(tile / (uint32_t)CT);
        });
        if (f.e < 0 || !on) return;
        e = f.e;
        r0 = f.row0;
        rows = (int)min((int64_t)BT, f.end - r0);
        c0 = BT * (int)(tile % (uint32_t)CT);
        R = e < p.E ? p.R : 0;
        const int64_t we = e < p.E ? e : 0;
        a = p.a + r0 * p.R;
        lda = p.R;
        as = p.as + r0;
        ldas = p.M;
        b = p.b + (we * p.C + c0) * p.R;
        bs = p.bs + we * p.bs_e + (int64_t)(c0 / 128) * p.bs_c;
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
        // the whole call is dropped where any offset is invalid (all of these
        // loads go out together)
        const int64_t o0 = p.offsets[e], o1 = p.offsets[e + 1];
        bool bad = p.offsets[0] != 0 || p.offsets[p.E] > p.M;
        for (int i = lane; i < p.E; i += 64) bad |= p.offsets[i + 1] < p.offsets[i];
        bad = __ballot(bad) != 0;
        if (t == 0 && threadIdx.x == 0) *p.err = bad ? 1 : 0;
        if (bad) return;
        R = o1 - o0;
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

    // Stage s into slot s & 1.
    auto issue = [&](int s) {
        const uint32_t slot = lds0 + (uint32_t)(s & 1) * (uint32_t)sizeof(Slot);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int row = 8 * (NG * wave + i) + (lane >> 3);
            const uint32_t ko = 128u * (uint32_t)s + 16u * (uint32_t)((lane & 7) ^ swz8(row));
            const uint32_t dst = slot + 1024u * (uint32_t)(NG * wave + i);
            dma_lds_r<16>(ra, (row < rows && ko < len) ? (uint32_t)row * ld + ko : OOB, dst + (uint32_t)offsetof(Slot, a));
            dma_lds_r<16, B_AUX>(rb, (row < cols && ko < len) ? (uint32_t)row * ld + ko : OOB, dst + (uint32_t)offsetof(Slot, b));
        }
        // (the same words twice where there are more waves than halves)
        const int h = BT == 128 ? wave & 1 : 0, row = s < nb ? 64 * h + lane : 0x7FFFFFFF;
        if (WGRAD && wave >= 2)
            dma_lds_r<4>(rsb, row < cols ? 4u * ((uint32_t)s * (uint32_t)ldbs + (uint32_t)row) : OOB,
                         slot + (uint32_t)offsetof(Slot, sb) + 256u * (uint32_t)h);
        else
            dma_lds_r<4>(rsa, row < rows ? 4u * ((uint32_t)s * (uint32_t)ldas + (uint32_t)row) : OOB,
                         slot + (uint32_t)offsetof(Slot, sa) + 256u * (uint32_t)h);
    };

    float4v acc[NG][NG];
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int j = 0; j < NG; ++j) acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};

    // Two stages are in flight: a wave takes all of a stage into registers, and
    // its slot is refilled with the stage after next before the products begin.
    issue(0);
    issue(1);
    for (int s = 0; s < nb; ++s) {
        wait_vmcnt<DMAS>();
        block_barrier();
        const uint32_t slot = (uint32_t)(s & 1) * (uint32_t)sizeof(Slot);
        const float sw = WGRAD ? 1.0f : bs[s * ldbs];
        int8v fa[NG], fb[NG];
        float4v sb[NG];
        float sc[NG];
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t c = (uint32_t)(16 * (NG * wn + j)), r = (uint32_t)(16 * (NG * wm + j));
            fb[j] = b128_frag(lds, slot + (uint32_t)offsetof(Slot, b) + 128u * c, lane);
            fa[j] = b128_frag(lds, slot + (uint32_t)offsetof(Slot, a) + 128u * r, lane);
            if constexpr (WGRAD)
                sb[j] = *(const __attribute__((address_space(3))) float4v*)(
                    lds + slot + (uint32_t)offsetof(Slot, sb) + 4u * (c + 4u * (uint32_t)(lane >> 4)));
            sc[j] = *(const __attribute__((address_space(3))) float*)(
                lds + slot + (uint32_t)offsetof(Slot, sa) + 4u * (r + (uint32_t)(lane & 15)));
        }
        wait_lgkmcnt0();
        block_barrier();
        issue(s + 2);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const float c = WGRAD ? sc[i] : sc[i] * sw;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const float4v d = b128_mfma(fb[j], fa[i]);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(WGRAD ? d[v] * sb[j][v] : d[v], c, acc[i][j][v]);
            }
        }
    }
    wait_vmcnt<0>();

    const __amdgpu_buffer_rsrc_t ro = make_rsrc(uniform_ptr(out), 0x7FFFFFFFu);
    const uint32_t ldo = (uint32_t)p.C * (OUT_F32 ? 4u : 2u);
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const int r = 16 * (NG * wm + i) + (lane & 15), c = 16 * (NG * wn + j) + 4 * (lane >> 4);
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

// 256 x CW output tiles: 8 waves, two per SIMD.  CW = 256: waves of 128 x 64 (NI =
// 8 groups of 16 rows; 4 where the tile has at most 128 rows); CW = 128: of 64 x 64.
// The stream of operands bounds the loop (its DMA alone takes 69% of the time,
// its matrix work alone 67%): a compute unit's first-level cache keeps a fixed
// number of lines in flight and an instruction that finds it full stalls its
// wave.  So two stages are in flight, and every wave issues its share of a
// stage's DMA spread over 18 MFMAs (over 9: 992 us in the case below, over 24:
// 909; all of it in four waves of the eight, over 9 / 24: 928 / 896, at twice
// the code and, for wgrad, more registers than there are).  A wave reads its
// fragments three row groups ahead: WIDE_X MFMAs before a stage's end its data
// is in registers (barrier X) and its slot is refilled with the stage after
// next, while the next one has until WIDE_Y MFMAs before the end (barrier Y) to
// land.  A sum waits two MFMAs for its product, so the vector units work beside
// the matrix cores: 16 of an MFMA's 32 cycles forward, 32 for wgrad.  B rows go
// to LDS in an order that leaves a lane 16 adjacent output columns.
// The last stage's row groups are stored as their sums end, beside its other
// products (after them: wgrad 1310 us, forward 891).
// Measured, 32768 rows x 4096 x 7168 over 32 experts: forward 886 us, 2.17
// PFLOP/s (128 x 128 tiles: 1220 us); dgrad 920 us, wgrad 1249 us; another card
// takes 3% longer.
constexpr int WT = 256;
template <int CW>
struct WideSlot {
    uint8_t a[WT * 128];
    uint8_t b[CW * 128];  // row 16 j + 4 q + v of each 64 holds output column 16 q + 4 j + v
    float sa[WT];
    float sb[WT];  // wgrad: by output column; else the 128-column blocks' scales
};
constexpr int WIDE_X = 12;  // MFMAs before a stage's end at which the slot's reads are over (barrier X)
constexpr int WIDE_Y = 8;   // and at which the next stage is needed (barrier Y)
constexpr int wide_dma(int CW) { return 5 + CW / 64; }  // DMA instructions per wave and stage
constexpr int WIDE_SPREAD = 18;  // MFMAs over which they go out (half as many in the loop of half as many MFMAs)

// DMA instruction n of a stage goes out behind the wide_due(n)th MFMA after X
// (counted through to the next stage); wide_sent(m): how many go before the mth.
template <int CW, int NI>
constexpr int wide_due(int n) { return n * (WIDE_SPREAD * NI / 8) / wide_dma(CW); }
template <int CW, int NI>
constexpr int wide_sent(int m) {
    int c = 0;
    for (int n = 0; n < wide_dma(CW); ++n) c += wide_due<CW, NI>(n) < m;
    return c;
}

template <bool OUT_F32, bool WGRAD, int CW>
__global__ __launch_bounds__(512, 1) void k_gemm_b128_wide(B128Args p) {
    extern __shared__ __align__(16) uint8_t s_wide[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int WM = CW == 256 ? 2 : 4;  // waves down the rows
    constexpr int WIDE_DMA = wide_dma(CW), BI = CW / 64;
    constexpr uint32_t WIDE_SLOT = sizeof(WideSlot<CW>);
    const int wm = wave & (WM - 1), wn = wave / WM;
    const int CT = (int)((p.C + CW - 1) / CW);
    // 32 consecutive tiles (4 row tiles x 8 column tiles) to an XCD at a time
    const int64_t t = (((int64_t)blockIdx.x >> 8) * 8 + (blockIdx.x & 7)) * 32 + ((blockIdx.x >> 3) & 31);
    int e, rows;
    int64_t r0, R;
    const uint8_t *a, *b;
    const float *as, *bs;
    int64_t lda, ldas, ldbs;
    char* out;
    int c0;
    if constexpr (!WGRAD) {
        const int64_t g = t / (4 * CT);
        const int l = (int)(t - g * 4 * CT);
        const RowTile f = find_row_tile<WT>(p, g * 4 + (l & 3), lane);
        if (f.e < 0) return;
        e = f.e;
        r0 = f.row0;
        rows = (int)min((int64_t)WT, f.end - r0);
        c0 = CW * (l >> 2);
        R = e < p.E ? p.R : 0;
        const int64_t we = e < p.E ? e : 0;
        a = p.a + r0 * p.R;
        lda = p.R;
        as = p.as + r0;
        ldas = p.M;
        b = p.b + (we * p.C + c0) * p.R;
        bs = p.bs + we * p.bs_e + (int64_t)(c0 / 128) * p.bs_c;
        ldbs = p.bs_b;
        out = static_cast<char*>(p.out) + (r0 * p.C + c0) * (OUT_F32 ? 4 : 2);
    } else {
        const int RT = (int)((p.R + WT - 1) / WT);
        if (t >= (int64_t)p.E * RT * CT) return;
        e = (int)(t / (RT * CT));
        const int l = (int)(t - (int64_t)e * RT * CT);
        const int g = l / (4 * CT), h = min(4, RT - 4 * g);
        const int ll = l - g * 4 * CT;
        r0 = WT * (4 * g + ll % h);
        c0 = CW * (ll / h);
        rows = (int)min((int64_t)WT, p.R - r0);
        // the whole call is dropped where any offset is invalid (all of these
        // loads go out together)
        const int64_t o0 = p.offsets[e], o1 = p.offsets[e + 1];
        bool bad = p.offsets[0] != 0 || p.offsets[p.E] > p.M;
        for (int i = lane; i < p.E; i += 64) bad |= p.offsets[i + 1] < p.offsets[i];
        bad = __ballot(bad) != 0;
        if (t == 0 && threadIdx.x == 0) *p.err = bad ? 1 : 0;
        if (bad) return;
        R = o1 - o0;
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
    rows = __builtin_amdgcn_readfirstlane(rows);
    const int cols = __builtin_amdgcn_readfirstlane((int)min((int64_t)CW, p.C - c0));
    const int nb = __builtin_amdgcn_readfirstlane((int)((R + 127) / 128));
    const uint32_t ld = __builtin_amdgcn_readfirstlane((uint32_t)lda);
    const uint32_t lsa = __builtin_amdgcn_readfirstlane((uint32_t)ldas), lsb = __builtin_amdgcn_readfirstlane((uint32_t)ldbs);
    // token columns are padded to whole blocks of zeros; k and n are not
    const uint32_t len = WGRAD ? (uint32_t)nb * 128u : __builtin_amdgcn_readfirstlane((uint32_t)R);
    // rows past the tile lie past the descriptors' ranges
    const __amdgpu_buffer_rsrc_t ra = rsrc_n(uniform_ptr(a), (uint32_t)rows * ld), rb = rsrc_n(uniform_ptr(b), (uint32_t)cols * ld);
    const __amdgpu_buffer_rsrc_t rsa = rsrc_n(uniform_ptr(as), 0x7FFFFFFFu), rsb = rsrc_n(uniform_ptr(bs), 0x7FFFFFFFu);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(s_wide));
    const __attribute__((address_space(3))) uint8_t* lds = (const __attribute__((address_space(3))) uint8_t*)(s_wide);

    // DMA of stage s into slot s & 1: instructions 2 i and 2 i + 1 move eight
    // rows of either operand (with 128 columns two more eight of A), the last
    // one the scales.
    // prep(s) sets the lane offsets of stage s: chunk (lane & 7) ^ swz8(row) of
    // the rows 8 i + lane / 8, even and odd i, or nowhere past the last stage.
    const int drow = lane >> 3;
    const uint32_t ch0 = 16u * (uint32_t)((lane & 7) ^ swz8(drow)), ch1 = 16u * (uint32_t)((lane & 7) ^ swz8(8 + drow));
    const uint32_t abase = (uint32_t)(32 * wave + drow) * ld;
    const uint32_t bbase = (uint32_t)((CW == 256 ? 64 * (wave >> 1) + 8 * (wave & 1) : 64 * (wave >> 2) + 4 * (wave & 3)) +
                                      16 * (drow >> 2) + (drow & 3)) * ld;
    // scales: waves 0..3 those of A, waves 4..7 those of B
    const int srow = 64 * (wave & 3) + lane;
    const bool sb_wave = wave >= 4;
    const __amdgpu_buffer_rsrc_t rsc = sb_wave ? rsb : rsa;
    const uint32_t lsc = sb_wave ? lsb : lsa;
    const uint32_t scoff = sb_wave ? (WGRAD ? (srow < cols ? 4u * (uint32_t)srow : OOB)
                                            : (srow < (cols + 127) / 128 ? 4u * (uint32_t)(srow * p.bs_c) : OOB))
                                   : (srow < rows ? 4u * (uint32_t)srow : OOB);
    const uint32_t scdst = (uint32_t)(sb_wave ? offsetof(WideSlot<CW>, sb) : offsetof(WideSlot<CW>, sa)) + 256u * (uint32_t)(wave & 3);
    uint32_t va[2], vb[2];
    auto prep = [&](int s) {
        const uint32_t k0 = 128u * (uint32_t)s + ch0, k1 = 128u * (uint32_t)s + ch1;
        va[0] = k0 < len ? abase + k0 : OOB;
        va[1] = k1 < len ? abase + k1 : OOB;
        vb[0] = k0 < len ? bbase + k0 : OOB;
        vb[1] = k1 < len ? bbase + k1 : OOB;
    };
    auto issue = [&](int s, int n) {
        const uint32_t slot = lds0 + (uint32_t)(s & 1) * WIDE_SLOT;
        if (n == WIDE_DMA - 1) {
            dma_lds_r<4>(rsc, s < nb ? scoff + 4u * (uint32_t)s * lsc : OOB, slot + scdst);
        } else if ((n & 1) && n < 2 * BI) {
            // LDS row CW / 8 wave + 8 i + lane / 8
            const int i = n >> 1;
            const uint32_t brow = (uint32_t)(CW == 256 ? 4 * (i >> 1) + 32 * (i & 1) : 32 * i);
            dma_lds_r<16>(rb, vb[i & 1] + brow * ld,
                          slot + (uint32_t)(16 * CW) * (uint32_t)wave + (uint32_t)offsetof(WideSlot<CW>, b) + 1024u * (uint32_t)i);
        } else {
            const int i = n < 2 * BI ? n >> 1 : n - BI;
            dma_lds_r<16>(ra, va[i & 1] + (uint32_t)(8 * i) * ld,
                          slot + 4096u * (uint32_t)wave + (uint32_t)offsetof(WideSlot<CW>, a) + 1024u * (uint32_t)i);
        }
    };

    prep(0);
#pragma unroll
    for (int n = 0; n < WIDE_DMA; ++n) issue(0, n);
    prep(1);
    const int lr = lane & 15, q = lane >> 4;
    const uint32_t fr = (uint32_t)(128 * lr + 16 * (q ^ swz8(lr)));
    const uint32_t ldo = (uint32_t)p.C * (OUT_F32 ? 4u : 2u);

    auto body = [&](auto NIC) {
        constexpr int NI = decltype(NIC)::value;
        constexpr int NM = 4 * NI, XM = NM - WIDE_X, YM = NM - WIDE_Y;
        const uint32_t fa = (uint32_t)offsetof(WideSlot<CW>, a) + (uint32_t)(wm * NI * 16 * 128) + fr, fa1 = fa ^ 64u;
        const uint32_t fb = (uint32_t)offsetof(WideSlot<CW>, b) + (uint32_t)(wn * 64 * 128) + fr, fb1 = fb ^ 64u;
        const uint32_t fsa = (uint32_t)offsetof(WideSlot<CW>, sa) + 4u * (uint32_t)(wm * NI * 16 + lr);
        const uint32_t fsb = (uint32_t)offsetof(WideSlot<CW>, sb) + (WGRAD ? 4u * (uint32_t)(64 * wn + 16 * q) : 4u * (uint32_t)(64 * wn / 128));
        auto frag = [&](uint32_t at, uint32_t at1) {
            const u32x4 x0 = *(const __attribute__((address_space(3))) u32x4*)(lds + at);
            const u32x4 x1 = *(const __attribute__((address_space(3))) u32x4*)(lds + at1);
            return int8v{(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3], (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
        };
        auto f32_at = [&](uint32_t at) { return *(const __attribute__((address_space(3))) float*)(lds + at); };
        float4v acc[NI][4], D[4], sB[4];
        int8v A[4], B[4];
        float sa[4], sw = 0.0f, sc = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            D[j] = sB[j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NI; ++i) acc[i][j] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
        }
        auto rdA = [&](int s, int i) {
            const uint32_t slot = (uint32_t)(s & 1) * WIDE_SLOT;
            A[i & 3] = frag(slot + fa + 2048u * (uint32_t)i, slot + fa1 + 2048u * (uint32_t)i);
            sa[i & 3] = f32_at(slot + fsa + 64u * (uint32_t)i);
        };
        auto rdB = [&](int s, int j) {
            const uint32_t slot = (uint32_t)(s & 1) * WIDE_SLOT + 2048u * (uint32_t)j;
            B[j] = frag(slot + fb, slot + fb1);
        };
        auto rdS = [&](int s, int j) {
            if constexpr (WGRAD)
                sB[j] = *(const __attribute__((address_space(3))) float4v*)(lds + (uint32_t)(s & 1) * WIDE_SLOT + fsb + 16u * (uint32_t)j);
        };
        auto add = [&](int i, int j, float c) {
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(WGRAD ? D[j][v] * sB[j][v] : D[j][v], c, acc[i][j][v]);
        };
        // stage 0 and the first instructions of stage 1 are in flight
#pragma unroll
        for (int n = 0; n < wide_sent<CW, NI>(NM - XM); ++n) issue(1, n);
        wait_vmcnt<wide_sent<CW, NI>(NM - XM)>();
        block_barrier();
#pragma unroll
        for (int i = 0; i < 3; ++i) rdA(0, i);
#pragma unroll
        for (int j = 0; j < 4; ++j) rdB(0, j);
        if constexpr (!WGRAD) sw = f32_at(fsb);
        rdS(0, 0);
        rdS(0, 1);
        // output of row group i, whose sums are complete
        const __amdgpu_buffer_rsrc_t ro = make_rsrc(uniform_ptr(out), 0x7FFFFFFFu);
        auto store_rows = [&](int i) {
            // Lanes 8 apart swap halves, so that an instruction covers whole lines
            // of 8 rows instead of every other 16 bytes of 16 rows (wgrad 1385 us
            // that way), and the stores can be non-temporal (1366 otherwise).
            const int r = wm * NI * 16 + 16 * i + (lr & 7), c = 64 * wn + 16 * q;
            const uint32_t up = r < rows && c < cols ? 0u : OOB, dn = r + 8 < rows && c < cols ? 0u : OOB;
            const uint32_t o = (uint32_t)r * ldo + (uint32_t)c * (OUT_F32 ? 4u : 2u) + (lr & 8 ? 16u : 0u);
            auto store = [&](const u32x4& x, const u32x4& y, uint32_t at) {  // 32 adjacent bytes
                u32x4 u, d;
    #pragma unroll
                for (int v = 0; v < 4; ++v) {
                    u[v] = (uint32_t)__builtin_amdgcn_update_dpp((int)x[v], (int)y[v], 0x128, 0xF, 0xC, false);
                    d[v] = (uint32_t)__builtin_amdgcn_update_dpp((int)y[v], (int)x[v], 0x128, 0xF, 0x3, false);
                }
                __builtin_amdgcn_raw_buffer_store_b128(u, ro, (int)(up | (o + at)), 0, OUT_STORE_NT);
                __builtin_amdgcn_raw_buffer_store_b128(d, ro, (int)(dn | (o + at + 8u * ldo)), 0, OUT_STORE_NT);
            };
            if constexpr (OUT_F32) {
    #pragma unroll
                for (int h = 0; h < 2; ++h)
                    store(__builtin_bit_cast(u32x4, acc[i][2 * h]), __builtin_bit_cast(u32x4, acc[i][2 * h + 1]), 32u * h);
            } else {
                u32x4 x[2];
    #pragma unroll
                for (int h = 0; h < 2; ++h)
                    x[h] = u32x4{pack_bf16x2(acc[i][2 * h][0], acc[i][2 * h][1]), pack_bf16x2(acc[i][2 * h][2], acc[i][2 * h][3]),
                                 pack_bf16x2(acc[i][2 * h + 1][0], acc[i][2 * h + 1][1]),
                                 pack_bf16x2(acc[i][2 * h + 1][2], acc[i][2 * h + 1][3])};
                store(x[0], x[1], 0u);
            }
        };
        // Slot m = 4 i + j: MFMA (i, j), then the sum of the MFMA two slots back,
        // so that no sum waits for the matrix core.  The last stage has nothing to
        // fetch or to read ahead; its row groups leave as they are done.
        auto stage = [&](int s, auto LASTC) {
            constexpr bool LAST = decltype(LASTC)::value != 0;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const float sc_i = WGRAD ? sa[i & 3] : sa[i & 3] * sw;
                if constexpr (!WGRAD && !LAST)
                    if (i == NI - 1) sw = f32_at((uint32_t)((s + 1) & 1) * WIDE_SLOT + fsb);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int m = 4 * i + j;
                    if (!LAST && m == XM) {
                        wait_lgkmcnt0();
                        block_barrier();
                    }
                    if constexpr (!LAST)
                        if (m == YM) {
                            wait_vmcnt<wide_sent<CW, NI>(YM - XM)>();
                            block_barrier();
                        }
                    const float4v d = b128_mfma(B[j], A[i & 3]);
                    // the sum two slots back
                    if (j >= 2) add(i, j - 2, sc_i);
                    else add((i + NI - 1) % NI, j + 2, sc);
                    D[j] = d;
                    if (i == 0 && j < 2) rdS(s, j + 2);
                    if (j == 0 && i + 3 < NI) rdA(s, i + 3);
                    if constexpr (LAST) {
                        if (i > 0 && j == 2) store_rows(i - 1);
                    } else {
                        if (i == NI - 1 && j >= 2) rdS(s + 1, j - 2);
                        // next stage's first fragments once their registers are free
                        if (m == YM) rdA(s + 1, 0);
                        if (m == YM + 2) rdA(s + 1, 1);
                        if (i == NI - 1) {
                            if (j == 0) rdA(s + 1, 2);
                            rdB(s + 1, j);
                        }
                        if (m == XM) prep(s + 2);
#pragma unroll
                        for (int n = 0; n < WIDE_DMA; ++n)
                            if (wide_due<CW, NI>(n) == (m >= XM ? m - XM : m - XM + NM)) issue(s + (m >= XM ? 2 : 1), n);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                sc = sc_i;
            }
        };
        for (int s = 0; s < nb - 1; ++s) stage(s, IC<0>{});
        if (nb > 0) {
            stage(nb - 1, IC<1>{});
            add(NI - 1, 2, sc);
            add(NI - 1, 3, sc);
        } else {
#pragma unroll
            for (int i = 0; i < NI - 1; ++i) store_rows(i);
        }
        store_rows(NI - 1);
        // nothing is on its way into LDS when the wave ends; the stores may be
        wait_vmcnt<(OUT_F32 ? 4 : 2) * NI>();
    };
    if constexpr (CW == 128) {
        body(IC<4>{});
    } else {
        if (rows > 128) body(IC<8>{});
        else body(IC<4>{});
    }
}

namespace {

constexpr int64_t kMaxOffset = (int64_t)1 << 31;  // 32-bit buffer offsets
constexpr int64_t MAX_GRID = (int64_t)1 << 24;    // workgroups of 256 threads (of 512: half as many)

bool al(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Most row tiles of TM rows that E experts and the rows past them can need.
int64_t max_row_tiles(int64_t M, int E, int TM) { return M / TM + (M < E + 1 ? M : E + 1); }

// Which form runs, by the call's sizes (us; tiles are counted from the average
// expert, whose last one counts half, as the host does not know the others):
//  - 32 x 32 tiles up to FEW_TILES tiles of 64 x 64, which would leave most compute
//    units idle, each at the rate of the lines its first-level cache has in flight: 8
//    rows over 2 experts of 304 x 5696 14 against 18, 219 over 19 of 416 x 5408 21
//    against 23, but 168 over 4 of 2912 x 5536 (184 tiles) 32 against 26.  wgrad up
//    to FEW_TILES_WGRAD: 25434 rows, 2 experts of 1040 x 224, 46 against 66, but 17129
//    over 5 of 160 x 1584 (375) 29 against 22.
//  - 64 x 64 tiles up to SOME_TILES of them: 862 rows over 3 experts of 2176 x 6128 40
//    against 49 of 128 x 128 tiles, 12113 over 3 of 160 x 2368 18 against 20, but 1140
//    over 10 of 2016 x 2512 (704) 31 against 27.  wgrad up to SOME_TILES_WGRAD: 28890
//    rows, 14 experts of 768 x 736, 59 against 86, but 2889 over 2 of 1056 x 5808
//    (3094) 47 against 43 and 39 of 256 x 256 tiles; below it a few long experts lose:
//    9852 rows of one of 3552 x 1488 101 against 89.
//  - 64 x 64 tiles also up to SOME_ROWS rows an expert, where most tiles are an expert's
//    last: 1024 rows over 32 experts of 2048 x 2048 35 (skewed; even 30) against 40 (32),
//    1536 over 48 of 1024 x 4096 53 (51) against 58 (54), 128 over 32 of 4096 x 7168 162
//    against 163, but 1024 214 (171) against 197 (167).  Their weight loads are
//    non-temporal where hardly a weight is read twice (up to STREAM_ROWS rows an expert),
//    the weights do not fit the last-level cache from one call to the next and their rows
//    are whole lines: 64 rows over 32 experts of 4096 x 7168 120 against 133, 128 146
//    against 162, 512 183 against 196, but 2048 304 against 260.
//  - wgrad beyond: 256 x 256 tiles.  256 x 128 ones where 128 x 128 ones need the
//    second place of some compute units and these only the first: 3001 rows over 12 experts of 1424
//    x 2000 22 against 29 and 30; 8 experts of 4096 x 7168, 1536 rows with the
//    routing's skew would be 93 against 75 and 83, hence the margin of 1/8; none with
//    FULL_ROWS rows an expert, where few tiles are an expert's last: 15921 rows of one
//    expert of 512 x 1952, 250 tiles, 21 against 29 and 33, 19273 over 3 of 304 x 3472,
//    229, 34 against 40 and 46, but 4051 over 12 of 1408 x 1184, 231, 25 against 20
//    and 21, and 7559 over 6 of 960 x 6912, just 256, 88 against 62.
//  - 128 x 128 tiles while about all of them run at once, two to a compute unit: 8
//    experts of 4096 x 7168, 1024 rows 49 to 63 (even experts to the routing's skew)
//    against 68 to 85, 2048 rows 81 to 113 against 99 to 86 (7/8 of those places from
//    CROWDED_ROWS rows an expert on, where the big tiles are fuller and the count is an
//    average: 3083 skewed rows over 28 experts of 1616 x 4160, 494 tiles, 70 against 51,
//    3434 over 17 of 1792 x 976, 483, 26 against 19, but 1536 even rows over 8 of 4096 x
//    7168, 512, 75 against 90; over random sizes of this kind the big tiles take 9%
//    less); and up to TILE_ROWS rows an expert, where most tiles are an expert's last:
//    32 experts of 4096 x 7168, 2048 rows 213 against 231.  Half as many where the
//    reduction is shorter than LONG_R, as the big tiles' stores go out beside products:
//    32 experts of 7168 x 2048, 2048 rows 107 to 118 against 99 to 113; 64 experts of
//    2048 x 2048, 2048 rows 48 to 56 against 45 to 60, 4096 rows 51 to 64 against 47 to 66.
//  - else 256 x 256 tiles.
constexpr int64_t FEW_TILES = 128, FEW_TILES_WGRAD = 256;
constexpr int64_t SOME_TILES = 576, SOME_TILES_WGRAD = 2048;
constexpr int64_t SOME_ROWS = 32;
constexpr int64_t TILE_ROWS = 64;
constexpr int64_t LONG_R = 4096;
constexpr int64_t STREAM_ROWS = 16;
constexpr int64_t TILES_AT_ONCE = 512;
constexpr int64_t CROWDED_ROWS = 96;
constexpr int64_t MID_AT_ONCE = 256;
constexpr int64_t FULL_ROWS = 512;
constexpr int64_t LAST_LEVEL_CACHE = (int64_t)256 << 20;

size_t plan_bytes(int E) { return (size_t)((plan_words(E + 1) * 4 + 255) / 256 * 256); }

template <class K>
bsq_status run(K kernel, int64_t grid, int threads, size_t lds, const B128Args& a, hipStream_t s) {
    if (grid >= MAX_GRID || grid * threads >= (int64_t)1 << 32) return BSQ_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(threads), lds, s, a);
    return hipGetLastError() == hipSuccess ? BSQ_OK : BSQ_ERR_HIP;
}

template <bool F32, bool WGRAD, int CW>
bsq_status launch_wide(const B128Args& a, hipStream_t s) {
    constexpr int lds = 2 * (int)sizeof(WideSlot<CW>);
    const int64_t ct = (a.C + CW - 1) / CW;
    const int64_t tiles = WGRAD ? (int64_t)a.E * ((a.R + WT - 1) / WT) * ct : (max_row_tiles(a.M, a.E, WT) + 3) / 4 * 4 * ct;
    static bool attr_set = false;  // idempotent; racing writers set the same value
    if (!attr_set) {
        if (hipFuncSetAttribute(reinterpret_cast<const void*>(&k_gemm_b128_wide<F32, WGRAD, CW>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess)
            return BSQ_ERR_HIP;
        attr_set = true;
    }
    return run(k_gemm_b128_wide<F32, WGRAD, CW>, (tiles + 255) / 256 * 256, 512, lds, a, s);
}

// Workgroups of k_gemm_b128_tile (forward: row tiles in groups of 8).
template <bool WGRAD, int BT>
int64_t tile_grid(const B128Args& a) {
    return (WGRAD ? a.E * ((a.R + BT - 1) / BT) : (max_row_tiles(a.M, a.E, BT) + 7) / 8 * 8) * ((a.C + BT - 1) / BT);
}

template <bool F32, bool WGRAD, int BT, int B_AUX>
bsq_status launch_tile(B128Args a, bool even, hipStream_t s) {
    a.even = even;
    return run(k_gemm_b128_tile<F32, WGRAD, BT, B_AUX>, tile_grid<WGRAD, BT>(a), 256, 0, a, s);
}

template <bool F32, bool WGRAD>
bsq_status launch_b128(const B128Args& a, hipStream_t s) {
    // tiles of TM x TN (forward: an expert's last one counts half)
    auto tiles = [&](int64_t TM, int64_t TN) {
        const int64_t ct = (a.C + TN - 1) / TN;
        return WGRAD ? a.E * ((a.R + TM - 1) / TM) * ct : (2 * (a.M / TM) + std::min(a.M, (int64_t)a.E)) * ct / 2;
    };
    const int64_t t64 = tiles(64, 64);
    // the smaller tiles in even shares where one scan of the experts counts them all (16
    // rows of one expert of 7168 x 2816 12 us against 21, 512 over 2 of 3584 x 4096 22
    // against 33; but 384 over 384 of 2048 x 1024 97 against 78, 1024 over 1024 of 512 x
    // 512 101 against 72)
    const bool even = a.E < 64;
    if (t64 <= (WGRAD ? FEW_TILES_WGRAD : FEW_TILES)) return launch_tile<F32, WGRAD, 32, 0>(a, even, s);
    if constexpr (WGRAD) {
        return t64 <= SOME_TILES_WGRAD ? launch_tile<F32, true, 64, 0>(a, even, s) : launch_wide<F32, true, 256>(a, s);
    } else {
        const int64_t t128 = tiles(128, 128);
        if (t64 <= SOME_TILES || (a.M <= SOME_ROWS * a.E && tile_grid<false, 64>(a) < MAX_GRID)) {
            const bool stream = a.M <= STREAM_ROWS * a.E && a.R % 128 == 0 && a.E * a.C * a.R > LAST_LEVEL_CACHE;
            return stream ? launch_tile<F32, false, 64, 2>(a, even, s) : launch_tile<F32, false, 64, 0>(a, even, s);
        }
        if (t128 > TILES_AT_ONCE / 2 && tiles(256, 128) <= (a.M < FULL_ROWS * a.E ? MID_AT_ONCE * 7 / 8 : MID_AT_ONCE))
            return launch_wide<F32, false, 128>(a, s);
        if (t128 > (a.M < CROWDED_ROWS * a.E ? TILES_AT_ONCE : TILES_AT_ONCE * 7 / 8) &&
            a.M > (a.R < LONG_R ? TILE_ROWS / 2 : TILE_ROWS) * a.E)
            return launch_wide<F32, false, 256>(a, s);
        return launch_tile<F32, false, 128, 0>(a, t128 <= TILES_AT_ONCE, s);
    }
}

template <bool WGRAD>
bsq_status launch_b128(const B128Args& a, bool f32, hipStream_t s) {
    return f32 ? launch_b128<true, WGRAD>(a, s) : launch_b128<false, WGRAD>(a, s);
}

}  // namespace
}  // namespace bsq

extern "C" {

size_t bsq_grouped_gemm_fp8b128_workspace_size(int32_t num_experts) {
    if (num_experts < 1 || num_experts > bsq::MAX_EXPERTS) return 0;
    return bsq::plan_bytes(num_experts);
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
    int32_t* err = static_cast<int32_t*>(workspace) + bsq::PLAN_ERR;
    const bsq::B128Args a{a_codes, a_scale, w_codes, w_scale, offsets, num_experts, m_total, k, n, 0,
                          nb * kb, kb, 1, y, err, 0};
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
                              nb * kb, 1, kb, dx, err, 0};
        const bsq_status st = bsq::launch_b128<false>(a, dx_dtype == BSQ_F32, stream);
        if (st != BSQ_OK) return st;
    }
    if (wg) {
        const bsq::B128Args a{dyt_codes, dyt_scale, xt_codes, xt_scale, offsets, num_experts, m_total, n, k, P,
                              0, 0, 0, dw, err, 0};
        return bsq::launch_b128<true>(a, dw_dtype == BSQ_F32, stream);
    }
    return BSQ_OK;
}

}  // extern "C"
