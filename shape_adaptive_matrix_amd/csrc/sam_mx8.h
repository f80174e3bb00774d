// Block-scaled 8-bit GEMM for gfx950 (OCP Microscaling formats).
//
// C[i][j] = sum over k of (2^(SA[i][k/32]-127) A[i][k]) * (2^(SB[j][k/32]-127) B[k][j]),
// with E4M3 or E5M2 element codes and E8M0 block scales, FP32 accumulation
// and output. Page "fix(fp4_gemm autotune) SM107 kernel family excluded from
// autotune candidates and heuristics update - #4856" is about choosing among
// tile variants of a block-scaled low-precision GEMM; it names no format,
// and these are the block-scaled formats gfx950's matrix cores implement.
//
// Storage: A is M rows and B is given as Bt, N rows of K codes (Bt[j][k] =
// B[k][j]); SA is M rows and SB N rows of K/32 scale codes; C is M rows of N
// floats. K % 32 == 0. Block scaling runs along K, so both operands and both
// scale arrays are K-contiguous.
//
//  * The scaled MFMA (32x32x64, f8f6f4 family) takes per lane 32 K values
//    of one row of A (one column of B) in two 16-byte halves, and one E8M0
//    scale per lane. Its two 32-value scale blocks are split over the lane
//    groups: block 0 is the low halves of lanes 0-31 and 32-63 (K 0..15 and
//    16..31), block 1 their high halves (K 32..47 and 48..63), and lane
//    group g supplies the scale of block g (established with one-hot
//    operands and distinct block scales). So lane group g, half h holds K
//    32 h + 16 g .. + 15 of a k-step, and each lane loads the scale of the
//    MX block 2 t + g of its own row or column: a scale is never broadcast.
//  * Global -> LDS: buffer loads that write LDS directly, 1 KB per wave
//    instruction, two stages of BK values of K. Out-of-range offsets write
//    zeros, so M, N and K tails need no other care.
//  * Both operands sit in LDS as K-contiguous rows of BK bytes, 16-byte
//    chunks XOR-swizzled by row, and a fragment is two 128-bit LDS reads (no
//    transposing read is needed for either operand).
//  * Scales (SDMA form, K % 128 == 0): a stage's BK/32 scale bytes of every
//    row travel with the stage's operands as 4-byte LDS loads (one wave
//    instruction moves one dword for each of 64 rows), and each lane reads
//    its rows' dwords from LDS once the stage has landed and extracts the
//    byte of its K block. Loading the scales per lane straight from memory
//    touches one cache line per row per instruction, which took more L1
//    lookups than the operands themselves and halved the throughput.
//    Byte form (other K, where the dwords would be misaligned): one byte
//    load per (MFMA block, K block) of the next stage, issued during the
//    current stage's first k-step. Either way the scale sits in byte 0 of
//    its register (scale byte select 0).
//  * One barrier per stage before its last k-step, as in the 16-bit kernel.
// No atomics and a fixed K order per output: repeated runs give the same
// bits.
#pragma once

#include "sam_dma.h"
#include "sam_internal.h"

namespace sam {
namespace mx8 {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned u8v __attribute__((ext_vector_type(8)));

template <int DT> struct Half;
template <> struct Half<DT_BF16> { typedef __bf16 T; };
template <> struct Half<DT_F16> { typedef _Float16 T; };

// EB: element bits, 8 (FA, FB: 0 E4M3, 1 E5M2) or 4 (FA = FB = 4, E2M1 packed
// two per byte, element 2 i in the low nibble). BK counts values of K.
// OUT: -1 C (or a split's partial sums) as compact FP32 rows; otherwise C (or a
// split's) of that type (DT_F32, DT_BF16, DT_F16) with row stride ldc, and Bt's
// rows of ldb values: K may be rounded up past them, for what A holds there
// are zeros and what Bt's next row holds are finite E2M1 values. The scales
// are K / 128 planes then, of a dword for every row (scale_rows, so that a
// plane starts on 16 bytes).
template <int FA, int FB, int BM, int BN, int WM, int WN, int BK, bool SDMA, int EB, int OUT = -1>
__global__ void __launch_bounds__(WM * WN * 64)
__attribute__((amdgpu_waves_per_eu(1, (160 * 1024 / (2 * (BM + BN) * (BK + 8))) * WM * WN / 4 > 0
                                           ? (160 * 1024 / (2 * (BM + BN) * (BK + 8))) * WM * WN / 4 : 1)))
gemm_mx8_kernel(GemmArgs args)
{
    using namespace dma;
    constexpr int NBUF = 2;
    constexpr int NW = WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int TM = WTM / 32, TN = WTN / 32;
    constexpr int ROW = BK * EB / 8;                   // bytes per LDS row
    constexpr int VPC = 128 / EB;                      // values of K per 16-byte chunk
    constexpr int RPB = EB == 8 ? 2 : 1;               // 128-bit LDS reads per MFMA operand block
    constexpr int CPR = ROW / 16;                      // 16-byte chunks per row
    constexpr int RPL = 64 / CPR;                      // rows per 1 KB wave load
    constexpr int RSW = CPR >= 16 ? 1 : 16 / CPR;      // rows sharing one 256-byte bank sweep
    constexpr int KSTEPS = BK / 64;                    // MFMA k-steps per stage
    constexpr int A_BYTES = BM * ROW, B_BYTES = BN * ROW;
    constexpr int SDW = BK / 128;                      // scale dwords per row per stage (SDMA)
    constexpr int S_BYTES = SDMA ? (BM + BN) * SDW * 4 : 0;   // [dword d][A rows, then Bt rows]; OUT: A's dwords, then Bt's
    constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES;
    constexpr int A_PW = A_BYTES / 1024 / NW, B_PW = B_BYTES / 1024 / NW;
    // Scale loads per stage: a dword of 64 rows each (OUT: four rows a lane).
    constexpr int SPA = BM * SDW / 256;                // of A (OUT)
    constexpr int SPL = SDMA ? (OUT >= 0 ? SPA + BN * SDW / 256 : (BM + BN) / 64 * SDW) : 0;
    constexpr int SPW = (SPL + NW - 1) / NW;           // ... per wave, at most
    constexpr int LPS = A_PW + B_PW + SPW;             // wave loads per stage (a wave may skip its last)
    // Stage loads by k-steps: the last of a stage issues loads 0 .. LATE - 1 of
    // the stage after next, the next stage's first LATE .. LATER - 1, its second
    // the rest. All of them in the last one (68 KB a k-step of a 256 x 256
    // E2M1 tile) take twice as long as its MFMAs, which wait behind them: E2M1
    // 4096 x 4096 x 11008 with the rounding 119 us, so 108; E4M3 8192^3 513
    // and 502.
    constexpr int LATE = !SDMA ? LPS : (EB == 4 ? LPS / 2 : LPS * 3 / 4);
    constexpr int LATER = KSTEPS > 2 && SDMA ? LATE + (LPS - LATE) / 2 : LPS;
    constexpr int NSB = TM + TN;                       // MFMA blocks whose scales a lane uses
    constexpr int NSR = SDMA ? SDW : KSTEPS;           // raw scale registers per block
    static_assert(EB == 8 || (EB == 4 && FA == 4 && FB == 4), "8-bit formats or E2M1");
    static_assert(OUT < 0 || SDMA, "planes of scale dwords");
    static_assert(ROW == 128 || ROW == 256, "K per stage: 128- or 256-byte rows");
    static_assert(BK % 128 == 0, "whole scale dwords per stage");
    static_assert(WTM % 32 == 0 && WTN % 32 == 0, "wave tile must be whole 32x32 blocks");
    static_assert(A_BYTES % (1024 * NW) == 0 && B_BYTES % (1024 * NW) == 0, "loads must split evenly over waves");
    static_assert(NBUF * STAGE <= 160 * 1024, "LDS");
    static_assert(LPS + (SDMA ? 0 : NSB * KSTEPS) < 64, "vmcnt range");
    static_assert(BM % 64 == 0 && BN % 64 == 0, "scale loads cover 64 rows");
    static_assert(OUT < 0 || (BM * SDW % 256 == 0 && BN * SDW % 256 == 0), "1 KB scale loads");
    static_assert(NBUF == 2, "the prologue fills two stages");
    static_assert(!SDMA || LATE <= A_PW + B_PW, "loads that every wave has");

    __shared__ __attribute__((aligned(1024))) unsigned char lds[NBUF * STAGE];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // uniform: scalar branches and selects
    int tm, tn, s;
    tile_coords(blockIdx.x, args, tm, tn, s);
    const int M = args.M, N = args.N, K = args.K;
    const int KB = K / 32;                             // scale codes per row
    const int RB = K * EB / 8;                         // bytes per operand row
    const int RBB = OUT >= 0 ? args.ldb * EB / 8 : RB; // of Bt: rows may be shorter than K (see OUT)
    const int m0 = tm * BM, n0 = tn * BN;
    const int kbeg = s * args.k_chunk;
    const int kend = min(K, kbeg + args.k_chunk);
    const int nk = kend > kbeg ? (kend - kbeg + BK - 1) / BK : 0;
    const int wm0 = (wave / WN) * WTM;
    const int wn0 = (wave % WN) * WTN;

    const i4 rA = rsrc_words(static_cast<const char*>(args.A) + (long long)m0 * RB, (long long)(M - m0) * RB);
    const i4 rB = rsrc_words(static_cast<const char*>(args.B) + (long long)n0 * RBB, (long long)(N - n0) * RBB);
    const __amdgpu_buffer_rsrc_t rSA = make_rsrc(args.sa + (long long)m0 * KB, (long long)(M - m0) * KB);
    const __amdgpu_buffer_rsrc_t rSB = make_rsrc(args.sb + (long long)n0 * KB, (long long)(N - n0) * KB);
    const i4 rSAw = rsrc_words(args.sa + (long long)m0 * KB, (long long)(M - m0) * KB);
    const i4 rSBw = rsrc_words(args.sb + (long long)n0 * KB, (long long)(N - n0) * KB);

    // Wave load q of stage `st`: q < A_PW fetch A rows, the rest Bt rows.
    // Lane l lands at dst + 16 l: row I * RPL + l / CPR, physical chunk
    // l % CPR, which holds logical chunk (K values 16 c .. 16 c + 15)
    // c = (l % CPR) ^ swizzle(row).
    // What depends on the lane is the same for all of a wave's loads (rows NW
    // RPL apart have the same swizzle), and there is no branch around them:
    // the loop stays one block, in which the MFMAs keep their places. (With a
    // branch for the K tail at every load the compiler moved all of a stage's
    // MFMAs behind its fragment reads: E2M1 4096 x 4096 x 11008 122 us.)
    static_assert(NW * RPL / RSW % CPR == 0, "one swizzle for a wave's rows");
    const int lrow0 = wave * RPL + lane / CPR;
    const int lchunk = (lane % CPR) ^ ((lrow0 / RSW) % CPR);
    const int lane_a = lrow0 * RB + lchunk * 16, lane_b = lrow0 * RBB + lchunk * 16;
    auto issue_one = [&](int st, int q) {
        const int k0 = kbeg + st * BK;
        unsigned char* buf = lds + (st % NBUF) * STAGE;
        if (q >= A_PW + B_PW) {
            // SDMA: scale load sq moves dword d of 64 consecutive rows (A
            // rows first, then Bt rows), i.e. scale codes 4 d .. 4 d + 3 of
            // the stage; dwords past the split's K and rows past M / N load
            // zero.
            const int sq = wave + (q - A_PW - B_PW) * NW;
            if (SPL % NW != 0 && sq >= SPL) return;
            if constexpr (OUT >= 0) {
                // Scales by dwords, each a plane of all rows: a lane takes
                // those of four. (From rows of scales every lane's dword lies
                // in a line of its own, 64 of them a load of 256 bytes: 4096 x
                // 11008 x 4096 without the rounding 105 us, from planes 99.)
                // Rows past M / N have any scales, for zeros.
                const bool is_a = sq < SPA;
                const int u = is_a ? sq : sq - SPA;
                const int at = u * 256 + lane * 4;               // row d R + r of the operand's R rows
                const int d = is_a ? at / BM : at / BN, r = is_a ? at % BM : at % BN;
                const long long rows = scale_rows(is_a ? M : N);
                const unsigned char* base = (is_a ? args.sa : args.sb) + (k0 / 128 * rows + (is_a ? m0 : n0)) * 4;
                const unsigned off = ((unsigned)d * (unsigned)rows + (unsigned)r) * 4;
                lds_load16(rsrc_words(base, ((K / 128 - k0 / 128) * rows - (is_a ? m0 : n0)) * 4),
                           lds_addr(buf + A_BYTES + B_BYTES + (is_a ? 0 : BM * SDW * 4) + u * 1024),
                           k0 + 128 * d < kend ? (int)off : kOOB);
            } else {
                constexpr int G = (BM + BN) / 64;              // 64-row groups
                const int d = sq / G, grp = sq % G;
                const bool is_a = grp * 64 < BM;
                const int r = grp * 64 - (is_a ? 0 : BM);      // first row of A or of Bt
                const int kb = k0 / 32 + 4 * d;
                const unsigned dst = lds_addr(buf + A_BYTES + B_BYTES + (d * (BM + BN) + grp * 64) * 4);
                const int first = kb * 32 < kend ? r * KB + kb : kOOB;
                lds_load4(is_a ? rSAw : rSBw, dst, (int)((unsigned)first + (unsigned)(lane * KB)));   // rows past M / N: past the record count
            }
            return;
        }
        // Rows past M (N) need no test: the panel's record count ends at row
        // M - m0 (N - n0), so their offsets read zero. K past the split's end
        // must be cut explicitly (it is the next split's, or the next row's).
        const bool is_a = q < A_PW;
        const int I = wave + (is_a ? q : q - A_PW) * NW;
        const bool in = lchunk * VPC < kend - k0;
        const unsigned at = (unsigned)((is_a ? q * RB : (q - A_PW) * RBB) * NW * RPL) + (unsigned)k0 * EB / 8;
        const unsigned off = (unsigned)(in ? (is_a ? lane_a : lane_b) : kOOB) + at;
        if (is_a)
            lds_load16(rA, lds_addr(buf + I * 1024), (int)off);
        else
            lds_load16(rB, lds_addr(buf + A_BYTES + I * 1024), (int)off);
    };

    // Scales of MFMA block b (b < TM: A block b, else Bt block b - TM): k-step
    // t uses K block 2 t + (lane >> 5) of the stage. sn holds the next
    // stage's raw registers, sc the current stage's:
    //  byte form: one code per k-step, in byte 0 (scale byte select 0);
    //  SDMA: the row's scale dword d (K blocks 4 d .. 4 d + 3) shifted down by
    //  8 (lane >> 5) bits, so that k-step t finds its code in byte 2 (t & 1)
    //  of register t >> 1 (scale byte select 2 (t & 1)).
    unsigned sc[NSB][NSR], sn[NSB][NSR];
    // Byte form: the next stage's codes straight from memory. Blocks past the
    // split's K, and rows past M / N, load zero (their elements are zero too).
    auto issue_scales = [&](int st, int b) {
        const int kb0 = (kbeg + st * BK) / 32;
#pragma unroll
        for (int t = 0; t < KSTEPS; ++t) {
            const int kb = kb0 + 2 * t + (lane >> 5);
            const bool kin = kb * 32 < kend;   // rows past M / N: past the record count
            if (b < TM) {
                const int row = wm0 + 32 * b + (lane & 31);
                sn[b][t] = __builtin_amdgcn_raw_buffer_load_b8(rSA, kin ? row * KB + kb : kOOB, 0, 0);
            } else {
                const int row = wn0 + 32 * (b - TM) + (lane & 31);
                sn[b][t] = __builtin_amdgcn_raw_buffer_load_b8(rSB, kin ? row * KB + kb : kOOB, 0, 0);
            }
        }
    };

    // SDMA: the scale dwords of block b's rows for the stage in `buf`.
    auto read_scales = [&](const unsigned char* buf, int b) {
        const int r = (b < TM ? wm0 + 32 * b : wn0 + 32 * (b - TM)) + (lane & 31);
#pragma unroll
        for (int d = 0; d < NSR; ++d) {
            const int at = OUT >= 0 ? (b < TM ? d * BM : SDW * BM + d * BN) : d * (BM + BN) + (b < TM ? 0 : BM);
            sn[b][d] = *reinterpret_cast<const unsigned*>(buf + A_BYTES + B_BYTES + (at + r) * 4);
        }
    };

    // Fragment reads, one 128-bit LDS read each; RPB per MFMA block: read
    // r < RPB TM is part r % RPB of A block r / RPB, the rest parts of Bt
    // blocks. A block i of k-step t sits in row wm0 + 32 i + (lane & 31).
    //  8-bit: half h holds K 64 t + 32 h + 16 (lane >> 5) .. + 15 of the
    //  stage (logical chunk 4 t + 2 h + (lane >> 5)), registers 4 h .. 4 h + 3:
    //  the instruction's scale block h is the h halves of both lane groups.
    //  4-bit: the lane holds K 64 t + 32 (lane >> 5) .. + 31 (logical chunk
    //  2 t + (lane >> 5)) in registers 0..3 (4..7 stay zero): for E2M1 the
    //  instruction applies lane group g's scale to all of lane group g's
    //  values, so each lane's share is exactly one MX block. (Both layouts
    //  were established with one-hot operands and distinct block scales.)
    auto read_one = [&](const unsigned char* buf, int t, int r, u8v (&fa)[TM], u8v (&fb)[TN]) {
        const bool is_a = r < RPB * TM;
        const int blk = is_a ? r / RPB : (r - RPB * TM) / RPB;
        const int h = r % RPB;
        const int row = (is_a ? wm0 : wn0) + 32 * blk + (lane & 31);
        u8v& f = is_a ? fa[blk] : fb[blk];
        const int lc = EB == 8 ? 4 * t + 2 * h + (lane >> 5) : 2 * t + (lane >> 5);
        const int c = lc ^ ((row / RSW) % CPR);
        const u4 v = *reinterpret_cast<const u4*>(buf + (is_a ? 0 : A_BYTES) + row * ROW + c * 16);
        if (h) f.hi = v; else f.lo = v;
    };

    v16f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    constexpr int NMF = TM * TN;                  // MFMAs per k-step
    constexpr int NRB = RPB * TN;                 // LDS reads of Bt fragments per k-step
    constexpr int RPS = (NRB + NMF - 1) / NMF;    // ... per MFMA slot
    constexpr int NRD = RPB * (TM + TN);          // all fragment reads of a k-step

    // One k-step: slot m issues MFMA m (A block m / TN, Bt block m % TN),
    // then the next k-step's Bt reads m * RPS .. (into the other Bt set),
    // then, after the last MFMA of A block i, the next k-step's reads of A
    // block i into the same registers (A fragments are single-buffered: each
    // is dead once its row of MFMAs has issued), then its share of the stage
    // loads q0 .. q1 - 1 or of the next stage's scales (first k-step:
    // global byte loads; last k-step, SDMA: LDS reads), evenly spread over
    // the slots.
    auto kstep = [&](u8v (&fa)[TM], const u8v (&fb)[TN], int t, const unsigned char* rbuf, int rt,
                     u8v (&nb)[TN], int load_stage, int q0, int q1, int scale_stage, int sread_stage) {
#pragma unroll
        for (int m = 0; m < NMF; ++m) {
            const int i = m / TN, j = m % TN;
            if constexpr (OUT >= 0) {
                // Operands exchanged: the block comes transposed, a lane's
                // values are four neighbours of a row of C each.
                if (t & 1)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        __builtin_bit_cast(v8i, fb[j]), __builtin_bit_cast(v8i, fa[i]), acc[i][j], FB, FA, 2,
                        (int)sc[TM + j][t >> 1], 2, (int)sc[i][t >> 1]);
                else
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        __builtin_bit_cast(v8i, fb[j]), __builtin_bit_cast(v8i, fa[i]), acc[i][j], FB, FA, 0,
                        (int)sc[TM + j][t >> 1], 0, (int)sc[i][t >> 1]);
            } else if constexpr (SDMA) {
                if (t & 1)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        __builtin_bit_cast(v8i, fa[i]), __builtin_bit_cast(v8i, fb[j]), acc[i][j], FA, FB, 2,
                        (int)sc[i][t >> 1], 2, (int)sc[TM + j][t >> 1]);
                else
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        __builtin_bit_cast(v8i, fa[i]), __builtin_bit_cast(v8i, fb[j]), acc[i][j], FA, FB, 0,
                        (int)sc[i][t >> 1], 0, (int)sc[TM + j][t >> 1]);
            } else {
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    __builtin_bit_cast(v8i, fa[i]), __builtin_bit_cast(v8i, fb[j]), acc[i][j], FA, FB, 0,
                    (int)sc[i][t], 0, (int)sc[TM + j][t]);
            }
#pragma unroll
            for (int r = m * RPS; r < (m + 1) * RPS; ++r)
                if (r < NRB) read_one(rbuf, rt, RPB * TM + r, fa, nb);
            if (j == TN - 1) {
#pragma unroll
                for (int h = 0; h < RPB; ++h) read_one(rbuf, rt, RPB * i + h, fa, nb);
            }
            if (load_stage >= 0) {
#pragma unroll
                for (int q = q0 + (m * (q1 - q0) + NMF - 1) / NMF; q < q0 + ((m + 1) * (q1 - q0) + NMF - 1) / NMF; ++q)
                    if (q < q1) issue_one(load_stage, q);
            }
            if (scale_stage >= 0) {
#pragma unroll
                for (int b = (m * NSB + NMF - 1) / NMF; b < ((m + 1) * NSB + NMF - 1) / NMF; ++b)
                    if (b < NSB) issue_scales(scale_stage, b);
            }
            if (SDMA && sread_stage >= 0) {
#pragma unroll
                for (int b = (m * NSB + NMF - 1) / NMF; b < ((m + 1) * NSB + NMF - 1) / NMF; ++b)
                    if (b < NSB) read_scales(lds + (sread_stage % NBUF) * STAGE, b);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto take_scales = [&]() {
#pragma unroll
        for (int b = 0; b < NSB; ++b)
#pragma unroll
            for (int d = 0; d < NSR; ++d) sc[b][d] = SDMA ? sn[b][d] >> (8 * (lane >> 5)) : sn[b][d];
    };

    u8v fa[TM], fb[2][TN];
    if constexpr (EB == 4) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[i].hi = u4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[0][j].hi = fb[1][j].hi = u4{0, 0, 0, 0};
    }
    // Stage 0 and what the loop does not load of stage 1; stage 0 and its
    // scales have landed when as many loads as that are left. Byte form:
    // stage 0 is drained completely, so that no scale load is still counted as
    // pending when the loop starts.
    if constexpr (!SDMA) {
#pragma unroll
        for (int b = 0; b < NSB; ++b) issue_scales(0, b);
    }
#pragma unroll
    for (int q = 0; q < LPS; ++q) issue_one(0, q);
    if constexpr (!SDMA) {
        wait_cnt<0, 15>();
        take_scales();
    }
#pragma unroll
    for (int q = 0; q < LATE; ++q) issue_one(1, q);
    if constexpr (SDMA) wait_cnt<LATE, 15>();
    barrier();
    if constexpr (SDMA) {
#pragma unroll
        for (int b = 0; b < NSB; ++b) read_scales(lds, b);
        take_scales();
    }
#pragma unroll
    for (int r = 0; r < NRD; ++r) read_one(lds, 0, r, fa, fb[0]);
    __builtin_amdgcn_sched_barrier(0);

    for (int k = 0; k < nk; ++k) {
        const unsigned char* cur = lds + (k % NBUF) * STAGE;
        const unsigned char* nxt = lds + ((k + 1) % NBUF) * STAGE;
        // k-steps 0 .. KSTEPS-2 of stage k, each reading the next k-step; the
        // first also loads stage k+1's scales (byte form), the first two the
        // rest of its operands (SDMA).
#pragma unroll
        for (int t = 0; t + 1 < KSTEPS; ++t)
            kstep(fa, fb[t & 1], t, cur, t + 1, fb[(t + 1) & 1], t < 2 && LATE < LPS ? k + 1 : -1, t ? LATER : LATE, t ? LPS : LATER, (!SDMA && t == 0) ? k + 1 : -1, -1);
        // Stage k fully read by this wave; stage k+1 and its scales landed.
        wait_cnt<0, 0>();
        barrier();
        // Last k-step of stage k: read k-step 0 of stage k+1 (and, SDMA, its
        // scales) and start to refill the slot stage k leaves with stage k + 2.
        constexpr int L = (KSTEPS - 1) & 1;
        kstep(fa, fb[L], KSTEPS - 1, nxt, 0, fb[L ^ 1], k + NBUF, 0, LATE, -1, SDMA ? k + 1 : -1);
        static_assert(L == 1, "an even number of k-steps per stage");
        take_scales();
    }
    wait_cnt<0, 0>();   // no LDS load may still be in flight when the workgroup ends

    const int lrow = lane & 31, lgrp = lane >> 5;
    if constexpr (OUT >= 0) {
        // Values to nearest even. Lane l holds row l % 32 of a block, columns
        // 8 g + 4 (l / 32) .. + 3 in registers 4 g .. 4 g + 3. Through LDS (32
        // of the wave's rows at a time, in the ring's place) to stores of 16
        // bytes, WTN columns of a row next to each other. (Stored from the
        // registers, 8 bytes a lane: 4096 x 11008 x 4096 99 us, so 92.)
        constexpr int ES = OUT == DT_F32 ? 4 : 2;
        constexpr int ROWB = WTN * ES + 16;                // a row in LDS, on banks of its own
        constexpr int LPR = WTN * ES / 16, RPI = 64 / LPR; // lanes to a row, rows an instruction
        static_assert(NW * 32 * ROWB <= NBUF * STAGE && LPR <= 64 && 64 % LPR == 0 && 32 % RPI == 0, "a block's rows of all waves in LDS");
        const int ld = args.ldc;
        char* outp = reinterpret_cast<char*>(args.out) + (s * args.part_stride + (long long)m0 * ld + n0) * ES;
        const __amdgpu_buffer_rsrc_t rC = make_rsrc(outp, ((long long)(M - m0 - 1) * ld + N - n0) * ES);
        // Rows on whole words are stored 16 bytes at a time, but for the last
        // columns.
        const bool words = ((long long)ld * ES % 4 == 0) && (reinterpret_cast<unsigned long long>(outp) & 3) == 0;
        unsigned char* mine = lds + wave * 32 * ROWB;
        barrier();   // all waves' last fragments are read
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    unsigned char* p = mine + lrow * ROWB + (32 * j + 8 * g + 4 * lgrp) * ES;
                    if constexpr (OUT == DT_F32) {
                        *reinterpret_cast<u4*>(p) = u4{__float_as_uint(acc[i][j][4 * g]), __float_as_uint(acc[i][j][4 * g + 1]),
                                                       __float_as_uint(acc[i][j][4 * g + 2]), __float_as_uint(acc[i][j][4 * g + 3])};
                    } else {
                        typedef typename Half<OUT>::T T;
                        typedef T T4 __attribute__((ext_vector_type(4)));
                        *reinterpret_cast<T4*>(p) = T4{(T)acc[i][j][4 * g], (T)acc[i][j][4 * g + 1], (T)acc[i][j][4 * g + 2],
                                                       (T)acc[i][j][4 * g + 3]};
                    }
                }
            // The wave's own rows: no barrier, its LDS accesses are in order.
            if (ES == 4 || words) {
#pragma unroll
                for (int t = 0; t < 32 / RPI; ++t) {
                    const int r = t * RPI + lane / LPR, c = lane % LPR * (16 / ES);
                    const u4 v = *reinterpret_cast<const u4*>(mine + r * ROWB + lane % LPR * 16);
                    const int row = wm0 + 32 * i + r, col = wn0 + c, left = N - n0 - col;
                    const int at = m0 + row < M ? (row * ld + col) * ES : kOOB;
                    __builtin_amdgcn_raw_buffer_store_b128(v, rC, left >= 16 / ES ? at : kOOB, 0, 0);
                    if (left > 0 && left < 16 / ES && at != kOOB) {
#pragma unroll
                        for (int e = 0; e < 16 / ES; ++e) {
                            if (e >= left) continue;
                            if constexpr (ES == 4)
                                __builtin_amdgcn_raw_buffer_store_b32(v[e], rC, at + 4 * e, 0, 0);
                            else
                                __builtin_amdgcn_raw_buffer_store_b16((unsigned short)(v[e / 2] >> (16 * (e % 2))), rC, at + 2 * e, 0, 0);
                        }
                    }
                }
            } else if constexpr (ES == 2) {   // rows that start inside a word: a value a lane
                constexpr int SPAN = WTN < 64 ? WTN : 64, RPV = 64 / SPAN;
#pragma unroll 8
                for (int t = 0; t < 32 / RPV * (WTN / SPAN); ++t) {
                    const int r = t / (WTN / SPAN) * RPV + lane / SPAN, c = t % (WTN / SPAN) * SPAN + lane % SPAN;
                    const int row = wm0 + 32 * i + r, col = wn0 + c;
                    __builtin_amdgcn_raw_buffer_store_b16(*reinterpret_cast<const unsigned short*>(mine + r * ROWB + c * 2), rC,
                                                          m0 + row < M && n0 + col < N ? (row * ld + col) * 2 : kOOB, 0, 0);
                }
            }
        }
        return;
    }
    float* outp = args.out + (long long)s * args.part_stride + (long long)m0 * N + n0;
    const __amdgpu_buffer_rsrc_t rC = make_rsrc(outp, ((long long)(M - m0) * N - n0) * 4);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int col = wn0 + 32 * j + lrow;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = wm0 + 32 * i + ((r >> 2) << 3) + (lgrp << 2) + (r & 3);
                const bool ok = m0 + row < M && n0 + col < N;
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][r]), rC,
                                                      ok ? (row * N + col) * 4 : kOOB, 0, 0);
            }
        }
    }
}

}  // namespace mx8
}  // namespace sam
