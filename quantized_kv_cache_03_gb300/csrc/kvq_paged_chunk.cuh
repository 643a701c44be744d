// kvq_paged_chunk.cuh -- attention of long query chunks over the paged cache
// (int8 K) on the 5th-generation tensor cores (tcgen05, accumulators in TMEM).
//
// The line of work and its split over persistent CTAs are those of
// kvq_paged_attn.cuh, in KV tiles of 128 positions of one 128-row tile of one kv
// head; under the causal mask a row tile counts the tiles its last row sees.
// One CTA per SM, 24 warps:
//   0-7   softmax, two groups of four warps, a thread one query row (its TMEM
//         lane): group g takes every other tile.  It quantizes half of the query
//         row into TMEM; of a tile it takes the row's maximum (first pass over
//         S), then p = 2^(s - m) in 32-position chunks, which overwrite S.  The
//         row's zero point m is handed from tile to tile through shared memory.
//         At the end of a piece each group writes half of O out.
//   8-11  K converters: k = code * scale as an fp16 high and low part.
//   12-19 V converters: v likewise, turned to [dim][position].
//   20    QK, 21 P.V: one thread each issues and waits.
//   22    walks the CTA's pieces of the line, hands them out as records, and
//         issues the bulk copies of the K parts of 64-position half tiles; 23 those
//         of the V parts.
// Tensor memory: S of two tiles (128 columns each), O, the query's high and low
// parts.  Shared memory: K and V operands of two half tiles.
// The two parts of a value hold it exactly at any scale: code * scale has 18 bits
// and is a multiple of 2^-24, fp16's least step (see code_hilo).
// QK: S = Qh Kh + Ql Kh + Qh Kl, the product of the low parts left out: within
// 2^-22 |q||k| of the exact sum of scaled integer block dots.  (The block dots
// themselves as four accumulators cost the softmax eight fp32 operations and a
// shared load per pair of scores and four times the tensor memory; that form
// measured 813 us on the 512-token chunk over 32768 positions.)
// P.V: KVQ_OUT_F16: P rounded to fp16 once (2^-11 at most of each weight, half
// of what the output's rounding adds up to), P.V_hi + P.V_lo; KVQ_OUT_F32: P in
// two fp16 parts, P_hi.V_hi + P_lo.V_hi + P_hi.V_lo (about 22 bits).
// m is raised only when a score would take P past 2^14, so after the first tile
// O is hardly ever rescaled; fp32 sums do not mind the range.
// The MMA cuts its sums off where fp32 would round them, so O falls short by
// 1e-9 to 5e-9 of itself per position (fp32 output, whose P.V takes three MMAs
// per 16 positions: 4.5e-5 after 32768, 1.7e-4 after 131072).  So every kCFlush
// tiles O joins sums in memory, in fp32, and starts again from zero.  Each softmax
// group has half of the columns: the group of the last tile does it while the
// other one makes the next P, and that one before it hands P over.  fp32 output,
// every 2 tiles: 1.3e-6 of the result's norm on a mixed batch (every 4 2.0e-6,
// every 8 3.4e-6; the same in PyTorch 1.4e-6), 321 us for it (309 every 4) and 620
// for the chunk named above (566); fp16 output, whose own rounding is 2e-4, every
// 64.  (One group for all columns, before its P: 319 and 669 us every 2.)
// Measured: that chunk, 32 heads on 8 kv heads, q4_0 V, fp16 output, takes 443 us
// (615 TFLOP/s counted as four times head_dim per visible pair of position and
// head), fp32 output 620.  The tensor pipe is active 56 % of the time; the K
// converters are busy 80 % of it, the softmax two thirds (fp32 output: four
// fifths), and the tile's chain QK, maximum, exponents, P.V hides only as far as
// two tiles of S in tensor memory allow.  Shared memory moves at 40 % of its rate.
// Every wait is bounded: a wait that gives up marks the CTA; the roles run out of
// waits in turn, drain what they issued and leave, and every row of the CTA's
// pieces is then written as NaN.
#pragma once

#include "kvq_paged.cuh"
#include "kvq_paged_line.cuh"
#include "kvq_prefill.cuh"

namespace kvq {

constexpr int kCM = kChunkRows;           // query rows per CTA: 128
constexpr int kCN = kChunkPositions;      // positions per KV tile: 128
constexpr int kCHalf = kCN / 2;           // positions per copied and converted half tile
constexpr int kCSub = kCHalf / kWTile;    // cache tiles per half
constexpr int kCChunk = 32;               // positions per softmax chunk
constexpr int kCKConv0 = 8, kCVConv0 = 12, kCQk = 20, kCPv = 21, kCKCopy = 22, kCVCopy = 23;
constexpr int kChunkWarps = 24, kChunkThreads = kChunkWarps * 32;
// Registers per thread: the launch gives every thread kCRegs (768 threads); the
// warpgroups then trade: 256 * 120 + 384 * 56 + 128 * 72 = 768 * 80.  (104, 64
// and 80: the softmax with fp32 output spills in its loop, 617 against 560 us on
// that chunk, with sums every 8 tiles.)
constexpr int kCRegs = 80, kCRegsSoft = 120, kCRegsConv = 56, kCRegsRest = 72;
static_assert(256 * kCRegsSoft + 384 * kCRegsConv + 128 * kCRegsRest <= kChunkThreads * kCRegs, "register shares");
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
constexpr int kCPieces = 4;              // piece records in flight
constexpr float kCShift = 8.0f, kCSlack = 6.0f;
// Tiles after which O is added to the rows' fp32 sums in memory and started
// afresh.
template <bool O16>
constexpr int kCFlush = O16 ? 64 : 2;

template <int VT>
struct ChunkCfg {
    using T = PageTile<VT, KVQ_K_I8>;
    // raw half tiles in flight: the K parts (codes, scales) and V parts of the
    // tile records in rings of their own, since K is converted ahead of V
    static constexpr int KPART = T::V_OFF, VPART = T::BYTES - T::V_OFF;
    static constexpr int RSK = VT == KVQ_V_Q4_0 ? 5 : 4, RSV = RSK, RAWK = kCSub * KPART, RAWV = kCSub * VPART;
    // K operand: 8-position row groups of 16 core matrices (8 positions x 8
    // dims), 160 bytes apart so that converter stores spread over the banks
    static constexpr int K_LBO = 160, K_SBO = 16 * K_LBO, KBUF = (kCHalf / 8) * K_SBO;
    // V operand [dim][position]: 8-dim row groups padded by 16 bytes, likewise
    static constexpr int V_SBO = (kCHalf / 8) * 128 + 16, VBUF = (kD / 8) * V_SBO;
    static constexpr int KH_OFF = 0, KL_OFF = KH_OFF + 2 * KBUF, VH_OFF = KL_OFF + 2 * KBUF, VL_OFF = VH_OFF + 2 * VBUF,
                         RAWK_OFF = VL_OFF + 2 * VBUF, RAWV_OFF = RAWK_OFF + RSK * RAWK;
    static constexpr int XM_OFF = RAWV_OFF + RSV * RAWV;              // fp32 [group][128]: a tile's m
    static constexpr int XE_OFF = XM_OFF + 2 * kCM * 4;             // float2 [group][128]: m, l at the end of a piece
    static constexpr int XS_OFF = XE_OFF + 2 * kCM * 8;             // float2 [group][128]: zero points of the sums, and of the O that joins them next
    static constexpr int REC_OFF = XS_OFF + 2 * kCM * 8;            // int [RSK], [RSV]: sub-tiles with a page
    static constexpr int OREC_OFF = REC_OFF + 48;                   // int [4 tiles][half]: the same, for the softmax
    static constexpr int PIECE_OFF = OREC_OFF + 32;                 // ChunkWalk [kCPieces], 64 bytes each
    static constexpr int BAR_OFF = PIECE_OFF + kCPieces * 64;
    // barriers; [i] by half, [g] by group (tile parity), [q] by lane quarter
    static constexpr int B_RAWK = 0, B_RAWV = B_RAWK + RSK, B_KF = B_RAWV + RSV, B_VF = B_KF + 2, B_PVD = B_VF + 2, B_FIN = B_PVD + 4,
                         B_PIECE = B_FIN + 2,                                               // one arrival: -, [i], [i], [g][i], -, -, and
                         B_M = B_PIECE + kCPieces, B_END = B_M + 8,                         // [g][q]
                         B_SFULL = B_END + 8,                                               // two, the QK thread and its commit: [g][i]
                         B_PREADY = B_SFULL + 4, B_KR = B_PREADY + 4, B_RAWKF = B_KR + 2,   // four warps: [g][i], [i], K ring, -
                         B_OFREE = B_RAWKF + RSK, B_VR = B_OFREE + 1, B_QR = B_VR + 2, B_RAWVF = B_QR + 1,   // eight warps: [i], -, V ring
                         B_PFREE = B_RAWVF + RSV, NBAR = B_PFREE + kCPieces;                  // all 23 roles
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;             // TMEM base, bad flag
    static constexpr int SMEM = MISC_OFF + 16;
    static_assert(KPART % 16 == 0 && VPART % 16 == 0 && RAWK_OFF % 128 == 0 && OREC_OFF % 8 == 0 && BAR_OFF % 8 == 0, "alignment");
    static_assert(RAWK_OFF < (1 << 18) && SMEM + 1024 <= 232448, "descriptor range, shared memory");
};

// 32 consecutive columns of this thread's TMEM lane; the wait passes the
// registers through, so that nothing reading them is moved ahead of it.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
                 "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32])
{
#define KVQ_R8(x, o) "+r"(x[o]), "+r"(x[o + 1]), "+r"(x[o + 2]), "+r"(x[o + 3]), "+r"(x[o + 4]), "+r"(x[o + 5]), "+r"(x[o + 6]), "+r"(x[o + 7])
    asm volatile("tcgen05.wait::ld.sync.aligned;" : KVQ_R8(r, 0), KVQ_R8(r, 8)::"memory");
    asm volatile("" : KVQ_R8(r, 16), KVQ_R8(r, 24)::"memory");
#undef KVQ_R8
}

// mbar_wait of a thread that runs alone: a loop of three instructions (the
// general one, inside a branch that one lane takes, slowed the MMA threads:
// 503 against 491 us on the chunk named above, as it was then).
template <uint32_t SPINS>
__device__ __forceinline__ bool mbar_wait_alone(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n .reg .pred p, q;\n .reg .u32 n;\n mov.u32 n, %3;\n"
                 "again:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra over;\n"
                 " sub.u32 n, n, 1;\n setp.ne.u32 q, n, 0;\n @q bra again;\n"
                 "over:\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity), "n"(SPINS)
                 : "memory");
    return done != 0;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(p));
    return p != 0;
}
// D (+)= A.B as umma_f16_ta_w, and its commit, by the one thread that runs this.
__device__ __forceinline__ void umma_ta_1(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void umma_commit_1(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Eight codes + 128 (two words) times the scale s (both halves).
__device__ __forceinline__ void u8x8_hilo(uint32_t w0, uint32_t w1, __half2 s, uint4 &hi, uint4 &lo)
{
    const __half2 st = __hmin2(s, __half2half2(__ushort_as_half(kTopScaleBits)));
    const __half2 k1152 = __half2half2(__ushort_as_half(0x6480));
    uint32_t r[4] = {__byte_perm(w0, 0x64646464u, 0x4140), __byte_perm(w0, 0x64646464u, 0x4342),
                     __byte_perm(w1, 0x64646464u, 0x4140), __byte_perm(w1, 0x64646464u, 0x4342)}, l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2 c = __hsub2(*reinterpret_cast<__half2 *>(&r[k]), k1152);
        code_hilo(*reinterpret_cast<const uint32_t *>(&c), st, s, r[k], l[k]);
    }
    hi = make_uint4(r[0], r[1], r[2], r[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// w[(k + r) % 4] = w[k].
__device__ __forceinline__ void turn4(uint32_t (&w)[4], int r)
{
    const bool one = r & 1, two = r & 2;
    const uint32_t a = one ? w[3] : w[0], b = one ? w[0] : w[1], c = one ? w[1] : w[2], d = one ? w[2] : w[3];
    w[0] = two ? c : a;
    w[1] = two ? d : b;
    w[2] = two ? a : c;
    w[3] = two ? b : d;
}

// A piece of the line, as the roles read it from shared memory.
struct ChunkWalk {
    int tiles;               // KV tiles with a visible position among those of the piece; negative: no more pieces
    int s0;                  // first KV tile
    int b, h, t0, n, L;      // sequence, kv head, first row and rows of the batch, length
    int lim0;                // last position the sequence's first row sees under the causal mask
    int gb, gsz, row0, R;    // query heads of the kv head, first row and rows of the tile
    int lim_hi;              // last position the tile's last row sees
    int slot;                // where the result goes: -1 out, else the CTA's slot of partials
};
// KV tiles a row tile counts for: those its last row sees (all, when the kv
// heads have query groups of different sizes), at least one.
__device__ __forceinline__ int chunk_tiles(const PagedAttnParams &p, int n, int L, int lim0, int rt)
{
    const int last = min(n - 1, (int)(((long long)rt * kCM + kCM - 1) / p.gmax));
    const int vis = p.causal && p.uniform ? min(L, lim0 + 1 + last) : L;
    return max(1, (vis + kCN - 1) / kCN);
}
__device__ __forceinline__ long long chunk_head_tiles(const PagedAttnParams &p, int n, int L, int lim0)
{
    const int n_rt = (int)(((long long)n * p.gmax + kCM - 1) / kCM);
    long long s = 0;
    for (int rt = 0; rt < n_rt; ++rt) s += chunk_tiles(p, n, L, lim0, rt);
    return s;
}

// Calls body(piece) for every piece of [pos, end) until it returns false;
// cuts: this CTA's entries.
template <typename F>
__device__ __forceinline__ void chunk_pieces(const PagedAttnParams &p, const LineStart &line, long long pos, long long end, long long per,
                                             PagedCut *cuts, F body)
{
    ChunkWalk w;
    w.b = line.b - 1;
    int rt = 0, n_rt = 0;
    bool fresh = true, first = true;
    const int H = p.pool.n_kv_heads;
    while (pos < end) {
        if (fresh) {
            do {
                ++w.b;
                seq_shape(p, w.b, w.t0, w.n, w.L, w.lim0);
            } while (!seq_mine(p, w.n));
            n_rt = (int)(((long long)w.n * p.gmax + kCM - 1) / kCM);
            w.h = rt = w.s0 = 0;
            if (first) {
                const long long per_head = chunk_head_tiles(p, w.n, w.L, w.lim0);
                w.h = (int)(line.off / per_head);
                long long x = line.off - w.h * per_head;
                for (;; ++rt) {
                    const int k = chunk_tiles(p, w.n, w.L, w.lim0, rt);
                    if (x < k) break;
                    x -= k;
                }
                w.s0 = (int)x;
                first = false;
            }
            fresh = false;
        }
        const int n_tl = chunk_tiles(p, w.n, w.L, w.lim0, rt), s1 = (int)min((long long)n_tl, w.s0 + (end - pos));
        w.gb = p.grp_begin[w.h];
        w.gsz = p.grp_begin[w.h + 1] - w.gb;
        w.row0 = rt * kCM;
        w.R = min(kCM, w.n * w.gsz - w.row0);
        if (w.R > 0) {
            w.lim_hi = p.causal ? w.lim0 + (w.row0 + w.R - 1) / w.gsz : w.L - 1;
            w.tiles = w.lim_hi < 0 ? 0 : max(0, min(s1, w.lim_hi / kCN + 1) - w.s0);
            w.slot = -1;
            if (w.s0 > 0 || s1 < n_tl) {
                w.slot = w.s0 == 0 ? 1 : 0;
                const long long x0 = pos - w.s0, c0 = x0 / per;
                cuts[w.slot] = PagedCut{w.b, w.h | rt << 8, (int)c0, (int)((x0 + n_tl - 1) / per - c0 + 1)};
            }
            if (!body(w)) return;
        }
        pos += s1 - w.s0;
        w.s0 = 0;
        if (++rt == n_rt) {
            rt = 0;
            if (++w.h == H) fresh = true;
        }
    }
}

// LOSE: the test flavour; CTA 0 leaves out the copy of the K (p.lose even) or V
// part of half tile p.lose / 2.
template <int VT, bool O16, bool LOSE = false>
__global__ void __launch_bounds__(kChunkThreads, 1) paged_chunk_kernel(const __grid_constant__ PagedAttnParams p)
{
    using C = ChunkCfg<VT>;
    using T = typename C::T;
    constexpr uint32_t kIdQK = umma_idesc_f16(kCM, kCHalf), kIdPV = umma_idesc_f16(kCM, kD);
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ LineStart line;
    __shared__ long long tmp[kChunkWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pshift = p.pool.pshift;

    pdl_wait();
    pdl_trigger();
    long long pos, per;
    line_find<kChunkThreads>(p, kChunkMinTiles,
                             [&](int n, int len, int lim0) { return (long long)p.pool.n_kv_heads * chunk_head_tiles(p, n, len, lim0); }, &line, tmp, pos, per);
    const long long end = min(pos + per, line.total);
    PagedCut *cuts = p.cuts + (size_t)blockIdx.x * 2;
    if (tid < 2) cuts[tid] = PagedCut{0, 0, 0, 0};
    if (pos >= end) return;   // block-uniform
    static_assert(sizeof(ChunkWalk) <= 64, "piece records");

    const uint32_t sbase = smem_u32(smem), bars = sbase + C::BAR_OFF;
    auto bar = [&](int k) { return bars + 8u * (uint32_t)k; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *bad = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    if (warp == kCQk) tmem_alloc(smem_u32(tmem_slot), 512);
    if (tid == 0) {
        *bad = 0;
        for (int k = 0; k < C::NBAR; ++k)
            mbar_init(bar(k), k < C::B_SFULL ? 1 : k < C::B_PREADY ? 2 : k < C::B_VR ? 4 : k < C::B_PFREE ? 8 : 23);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tO = tmem + 2 * kCN, tQ = tO + kD;   // S of group g at 128 g; Q high parts, then low parts

    const bool loser = LOSE && blockIdx.x == 0;
    constexpr uint32_t kSpins = LOSE ? kLostCopySpins : kMbarSpins;
    auto give_up = [&]() {   // one thread of a role; the others run out of waits in turn
        if (atomicExch(const_cast<int *>(bad), 1) == 0) atomicAdd(p.timeouts, 1u);
    };
    auto wwait = [&](int k, uint32_t parity) {   // by a whole warp
        if (__all_sync(0xffffffffu, mbar_wait(bar(k), parity, kSpins))) return true;
        if (lane == 0) give_up();
        return false;
    };
    auto wait1 = [&](int k, uint32_t parity) {   // by one thread
        if (mbar_wait_alone<kSpins>(bar(k), parity)) return true;
        give_up();
        return false;
    };
    auto join_roles = [] { asm volatile("bar.sync 1, %0;" ::"n"(kChunkThreads) : "memory"); };   // every role has left its loop

    // Calls body(piece) for the pieces in turn; one = the calling thread is alone.
    auto pieces = [&](bool one, auto body) {
        for (int k = 0;; ++k) {
            const int e = k % kCPieces;
            if (!(one ? wait1(C::B_PIECE + e, (k / kCPieces) & 1) : wwait(C::B_PIECE + e, (k / kCPieces) & 1))) return;
            const ChunkWalk &w = *reinterpret_cast<const ChunkWalk *>(smem + C::PIECE_OFF + 64 * e);
            if (w.tiles < 0 || !body(w, k)) return;
            if (!one) __syncwarp();
            if (one || lane == 0) mbar_arrive(bar(C::B_PFREE + e));
        }
    };

    // (each share is set inside its own branch: where branches with different
    // shares join, the compiler would hold all of them to the smallest)
    if (warp >= kCQk) {
    regs_dec<kCRegsRest>();
    if (warp == kCKCopy || warp == kCVCopy) {
        // ================= bulk copies: a warp for the K parts, one for the V parts; the first
        // also walks the pieces and hands them out =================
        const bool kside = warp == kCKCopy;
        const int rs = kside ? C::RSK : C::RSV, part = kside ? C::KPART : C::VPART;
        const int b_full = kside ? C::B_RAWK : C::B_RAWV, b_free = kside ? C::B_RAWKF : C::B_RAWVF;
        const uint32_t raw = sbase + (kside ? C::RAWK_OFF : C::RAWV_OFF);
        int *rec = reinterpret_cast<int *>(smem + C::REC_OFF) + (kside ? 0 : C::RSK);
        int issued = 0, st = 0, ph = 0;   // halves so far, the ring's slot and its phase
        const size_t page_bytes = ((size_t)p.pool.n_kv_heads << (pshift - 4)) * T::BYTES;
        auto copy_piece = [&](const ChunkWalk &w) {
            const int *bt = p.block_table + (size_t)w.b * p.table_stride;
            const uint8_t *head = p.pool.data + ((size_t)w.h << (pshift - 4)) * T::BYTES + (kside ? 0 : T::V_OFF);
            const int n_half = 2 * w.tiles;
            const uint8_t *src = nullptr;   // lane l: sub-tile l % 4 of half t + l / 4, for eight halves at a time
            for (int t = 0; t < n_half; ++t, ++issued) {
                if ((t & 7) == 0) {
                    const int x = w.s0 * kCN + (t + (lane >> 2)) * kCHalf + (lane & 3) * kWTile;
                    const int page = t + (lane >> 2) < n_half && x < w.L ? bt[x >> pshift] : -1;
                    src = page >= 0 && page < p.pool.n_pages ? head + page * page_bytes + ((x & ((1 << pshift) - 1)) >> 4) * T::BYTES : nullptr;
                }
                if (issued >= rs && !wwait(b_free + st, ph ^ 1)) return false;
                const int ok = (int)(__ballot_sync(0xffffffffu, src != nullptr) >> (4 * (t & 7))) & 15;
                const uint32_t full = bar(b_full + st);
                if (lane == 0) rec[st] = ok;
                __syncwarp();   // the record before the arrival that publishes it
                mbar_arrive_expect_tx_w(full, __popc(ok) * part);
                if ((lane >> 2) == (t & 7) && src && !(LOSE && loser && issued == p.lose >> 1 && (p.lose & 1) == (kside ? 0 : 1)))
                    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                     raw + (st * kCSub + (lane & 3)) * part),
                                 "l"(src), "r"(part), "r"(full)
                                 : "memory");
                __syncwarp();
                if (++st == rs) {
                    st = 0;
                    ph ^= 1;
                }
            }
            return true;
        };
        if (kside) {
            int k = 0;
            auto put = [&](const ChunkWalk &w) {
                const int e = k % kCPieces;
                if (k >= kCPieces && !wwait(C::B_PFREE + e, (k / kCPieces - 1) & 1)) return false;
                if (lane == 0) {
                    *reinterpret_cast<ChunkWalk *>(smem + C::PIECE_OFF + 64 * e) = w;
                    mbar_arrive(bar(C::B_PIECE + e));
                }
                ++k;
                return w.tiles <= 0 || copy_piece(w);
            };
            chunk_pieces(p, line, pos, end, per, cuts, put);
            ChunkWalk last = {};
            last.tiles = -1;
            put(last);
        } else {
            pieces(false, [&](const ChunkWalk &w, int) { return copy_piece(w); });
        }
        for (int k = max(0, issued - rs); k < issued; ++k)   // copies in flight
            if (!(LOSE && loser && k == p.lose >> 1 && (p.lose & 1) == (kside ? 0 : 1))) mbar_wait(bar(b_full + k % rs), (k / rs) & 1);
    } else if (warp == kCQk || warp == kCPv) {
        // ================= MMAs: one thread each =================
        if (elect_one()) {
            int j = 0, piece = 0, joins = 0;   // tiles, pieces with any, and starts of O from zero within pieces so far
            if (warp == kCQk) {
                uint64_t dKH[2], dKL[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    dKH[i] = umma_desc(sbase + C::KH_OFF + i * C::KBUF, C::K_LBO, C::K_SBO);
                    dKL[i] = umma_desc(sbase + C::KL_OFF + i * C::KBUF, C::K_LBO, C::K_SBO);
                }
                pieces(true, [&](const ChunkWalk &w, int) {
                    if (w.tiles == 0) return true;
                    if (!wait1(C::B_QR, piece & 1)) return false;
                    ++piece;
                    for (int k = 0; k < w.tiles; ++k, ++j) {
                        const int g = j & 1;
                        const uint32_t d = tS + kCN * g;
#pragma unroll 1
                        for (int i = 0; i < 2; ++i) {
                            // this half of P(j - 2) is used up, and K is there
                            if (j >= 2 && !wait1(C::B_PVD + 2 * g + i, ((j - 2) >> 1) & 1)) return false;
                            if (!wait1(C::B_KR + i, j & 1)) return false;
                            const uint64_t kh = i ? dKH[1] : dKH[0], kl = i ? dKL[1] : dKL[0];
                            tc_fence_after();
                            // the small terms first: the sum is cut off at each addition, by little while it is small
#pragma unroll
                            for (int term = 0; term < 3; ++term)   // Ql Kh, Qh Kl, Qh Kh
#pragma unroll
                                for (int ks = 0; ks < kD / 16; ++ks) {
                                    const uint64_t o = (uint64_t)(2 * ks * (C::K_LBO / 16));
                                    umma_ta_1(d + kCHalf * i, tQ + (term == 0 ? kD / 2 : 0) + 8 * ks, (term == 1 ? kl : kh) + o, kIdQK,
                                              term > 0 || ks > 0);
                                }
                            umma_commit_1(bar(C::B_KF + i));
                            umma_commit_1(bar(C::B_SFULL + 2 * g + i));
                            mbar_arrive(bar(C::B_SFULL + 2 * g + i));   // hands on what the converters published
                        }
                    }
                    return true;
                });
            } else {
                uint64_t dVH[2], dVL[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    dVH[i] = umma_desc(sbase + C::VH_OFF + i * C::VBUF, 128, C::V_SBO);
                    dVL[i] = umma_desc(sbase + C::VL_OFF + i * C::VBUF, 128, C::V_SBO);
                }
                pieces(true, [&](const ChunkWalk &w, int) {
                    for (int k = 0; k < w.tiles; ++k, ++j) {
                        const int g = j & 1;
                        // O starts from zero: the group of this tile has read its half of it (it says P is ready
                        // after that), the other group says so here
                        if (k > 0 && k % kCFlush<O16> == 0 && !wait1(C::B_OFREE, joins++ & 1)) return false;
#pragma unroll 1
                        for (int i = 0; i < 2; ++i) {
                            if (!wait1(C::B_VR + i, j & 1) || !wait1(C::B_PREADY + 2 * g + i, (j >> 1) & 1)) return false;
                            tc_fence_after();
                            const uint64_t vh = i ? dVH[1] : dVH[0], vl = i ? dVL[1] : dVL[0];
#pragma unroll
                            for (int ks = 0; ks < kCHalf / 16; ++ks) {
                                // chunk of 32 positions: high parts in its first 16 columns, low parts after
                                const uint32_t ph = tS + kCN * g + kCChunk * (2 * i + (ks >> 1)) + 8 * (ks & 1), pl = ph + kCChunk / 2;
                                const uint64_t o = (uint64_t)(16 * ks);
                                umma_ta_1(tO, ph, vh + o, kIdPV, (k % kCFlush<O16> || i > 0 || ks > 0) ? 1u : 0u);
                                if (!O16) umma_ta_1(tO, pl, vh + o, kIdPV, 1u);
                                umma_ta_1(tO, ph, vl + o, kIdPV, 1u);
                            }
                            umma_commit_1(bar(C::B_VF + i));
                            umma_commit_1(bar(C::B_PVD + 2 * g + i));
                        }
                    }
                    return true;
                });
            }
            // everything issued here is done before TMEM is freed
            const int fin = warp == kCQk ? C::B_FIN : C::B_FIN + 1;
            umma_commit_1(bar(fin));
            if (!mbar_wait_alone<kMbarSpins>(bar(fin), 0)) give_up();   // (the general wait here: 466 instead of 448 us on that chunk)
        }
        __syncwarp();
    }
    join_roles();
    } else if (warp >= kCKConv0) {
    regs_dec<kCRegsConv>();
    if (warp < kCVConv0) {
        // ================= K converters =================
        const int i = warp - kCKConv0;   // 16-byte chunk i of each cache tile: one position's codes of two blocks
        const int u = 8 * (i >> 1) + (lane >> 2), dg = 8 * (i & 1) + (lane & 3);
        const int soff = T::KS_OFF + (u >> 1) * 16 + 8 * (i & 1);   // both blocks' scales of positions u & ~1, u | 1
        const uint32_t mine = u & 1 ? 0x3232u : 0x1010u;
        int hh = 0;
        pieces(false, [&](const ChunkWalk &w, int) {
            for (int t = 0; t < 2 * w.tiles; ++t, ++hh) {
                const int st = hh % C::RSK, ob = hh & 1, j = hh >> 1;
                if (!wwait(C::B_RAWK + st, (hh / C::RSK) & 1) || (j >= 1 && !wwait(C::B_KF + ob, (j - 1) & 1))) return false;
                const uint8_t *raw = smem + C::RAWK_OFF + st * C::RAWK;
                uint8_t *kh = smem + C::KH_OFF + ob * C::KBUF + (u / 8) * C::K_SBO + (u % 8) * 16 + dg * C::K_LBO, *kl = kh + (C::KL_OFF - C::KH_OFF);
                uint4 va[kCSub];   // every load first: this role is the busiest (fp16 output, the chunk named above 460 -> 450 us)
                uint2 sa[kCSub];
#pragma unroll
                for (int q = 0; q < kCSub; ++q) {
                    va[q] = *reinterpret_cast<const uint4 *>(raw + q * C::KPART + i * 512 + lane * 16);
                    sa[q] = *reinterpret_cast<const uint2 *>(raw + q * C::KPART + soff);
                }
#pragma unroll
                for (int q = 0; q < kCSub; ++q) {
                    const uint4 v = va[q];
                    const uint2 sc = sa[q];
                    const uint32_t s0 = __byte_perm(sc.x, 0u, mine), s1 = __byte_perm(sc.y, 0u, mine);
                    uint4 hi, lo;
                    u8x8_hilo(v.x, v.y, *reinterpret_cast<const __half2 *>(&s0), hi, lo);
                    *reinterpret_cast<uint4 *>(kh + 2 * q * C::K_SBO) = hi;
                    *reinterpret_cast<uint4 *>(kl + 2 * q * C::K_SBO) = lo;
                    u8x8_hilo(v.z, v.w, *reinterpret_cast<const __half2 *>(&s1), hi, lo);
                    *reinterpret_cast<uint4 *>(kh + 2 * q * C::K_SBO + 4 * C::K_LBO) = hi;
                    *reinterpret_cast<uint4 *>(kl + 2 * q * C::K_SBO + 4 * C::K_LBO) = lo;
                }
                if (i == 0 && lane == 0)
                    reinterpret_cast<int *>(smem + C::OREC_OFF)[2 * (j & 3) + ob] = reinterpret_cast<const int *>(smem + C::REC_OFF)[st];
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::B_KR + ob));
                    mbar_arrive(bar(C::B_RAWKF + st));
                }
            }
            return true;
        });
    } else {
        // ================= V converters =================
        const int cw = warp - kCVConv0, q = cw >> 1, half = cw & 1;   // this warp: 8 positions of sub-tile q
        const int g = lane & 7, bb = lane >> 3;                      // this thread: block bb, code column g: four dims
        int hh = 0;
        pieces(false, [&](const ChunkWalk &w, int) {
            for (int t = 0; t < 2 * w.tiles; ++t, ++hh) {
                const int st = hh % C::RSV, ob = hh & 1, j = hh >> 1;
                if (!wwait(C::B_RAWV + st, (hh / C::RSV) & 1) || (j >= 1 && !wwait(C::B_VF + ob, (j - 1) & 1))) return false;
                const uint8_t *tv = smem + C::RAWV_OFF + st * C::RAWV + q * C::VPART, *ts = tv + (T::VS_OFF - T::V_OFF) + 4 * half * 16 + 4 * bb;
                const int ok = reinterpret_cast<const int *>(smem + C::REC_OFF)[C::RSK + st];
                const int x = w.s0 * kCN + t * kCHalf, p0 = x + kWTile * q + 8 * half;
                const bool full = ok == 15 && x + kCHalf - 1 <= w.lim_hi;
                uint32_t hi[4][4], lo[4][4];   // [dim of four][position pair]
                // The words of position pair c are 64 bytes apart over the columns, so the columns begin
                // with different pairs (a warp's load in one wavefront, or two for q8_0, instead of four
                // and eight) and the words are put in order afterwards.
                uint32_t vw[4], vx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = (k + (g >> 1)) & 3;
                    vx[k] = 0u;
                    if (VT == KVQ_V_Q4_0) {
                        vw[k] = *reinterpret_cast<const uint32_t *>(tv + half * 512 + (4 * g + c) * 16 + 4 * bb);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2 *>(tv + (2 * half + (bb >> 1)) * 512 + (4 * g + c) * 16 + 8 * (bb & 1));
                        vw[k] = v.x;
                        vx[k] = v.y;
                    }
                }
                turn4(vw, g >> 1);
                if (VT == KVQ_V_Q8_0) turn4(vx, g >> 1);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t dw = *reinterpret_cast<const uint32_t *>(ts + 16 * c);   // scales of positions 2c, 2c + 1
                    if (!full) {   // 0 where no row sees them
                        const bool live = ok >> q & 1;
                        dw &= (live && p0 + 2 * c <= w.lim_hi ? 0xffffu : 0u) | (live && p0 + 2 * c + 1 <= w.lim_hi ? 0xffff0000u : 0u);
                    }
                    const __half2 d2 = *reinterpret_cast<const __half2 *>(&dw);
                    // (q4_0: 8 * 8188 is fp16's largest number)
                    const __half2 dt = VT == KVQ_V_Q4_0 ? d2 : __hmin2(d2, __half2half2(__ushort_as_half(kTopScaleBits)));
                    uint32_t r[2][2];
                    v_codes<VT>(vw[c], vx[c], r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) code_hilo(r[e >> 1][e & 1], dt, d2, hi[e][c], lo[e][c]);
                }
                uint8_t *vh = smem + C::VH_OFF + ob * C::VBUF + cw * 128, *vl = vh + (C::VL_OFF - C::VH_OFF);
#pragma unroll
                for (int e = 0; e < 4; ++e) {   // r[h2][half] of v_codes: dim v_dim(2 bb + h2, g) + half
                    const int dim = v_dim<VT>(2 * bb + (e >> 1), g) + (e & 1);
                    const int o = (dim >> 3) * C::V_SBO + (dim & 7) * 16;
                    *reinterpret_cast<uint4 *>(vh + o) = make_uint4(hi[e][0], hi[e][1], hi[e][2], hi[e][3]);
                    *reinterpret_cast<uint4 *>(vl + o) = make_uint4(lo[e][0], lo[e][1], lo[e][2], lo[e][3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::B_VR + ob));
                    mbar_arrive(bar(C::B_RAWVF + st));
                }
            }
            return true;
        });
    }
    join_roles();
    } else {
        // ================= softmax: one query row per thread =================
        regs_inc<kCRegsSoft>();
        const int grp = warp >> 2, quarter = warp & 3;
        const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
        const int row = 32 * quarter + lane;
        const uint32_t tSg = tS + lane_base + kCN * grp;
        float *xm = reinterpret_cast<float *>(smem + C::XM_OFF);
        float2 *xe = reinterpret_cast<float2 *>(smem + C::XE_OFF);
        float2 *xs = reinterpret_cast<float2 *>(smem + C::XS_OFF) + grp * kCM + row;   // .x: the sums' zero point, .y: that of the O to join them
        // the scale's sign is in Q; a scale of 0 stays finite times -inf
        const float cs = fmaxf(fabsf(p.qk_scale_log2), 1e-30f);
        // the row's sums in memory, [dims / 4][row]: this group's half of them, which no other thread touches
        auto sums = [&]() { return reinterpret_cast<float4 *>(p.sums + (size_t)blockIdx.x * kChunkSums) + (kD / 8) * grp * kCM + row; };
        int j = 0, ends = 0;
        bool lost = false;
        pieces(false, [&](const ChunkWalk &w, int) {
            const bool whole = w.slot < 0;
            const bool row_ok = row < w.R;
            const int tok = row_ok ? (w.row0 + row) / w.gsz : 0, head = row_ok ? p.grp_q[w.gb + (w.row0 + row) % w.gsz] : 0;
            const int lim = row_ok ? (p.causal ? w.lim0 + tok : w.L - 1) : -1;
            float m = -INFINITY, l = 0.f;
            if (w.tiles > 0 && !lost) {
                // ---- blocks 2 grp, 2 grp + 1 of this row: int8 rule, q in two fp16 parts into TMEM ----
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (size_t)(w.t0 + tok) * p.q_stride + (size_t)head * kD);
                const float sgn = p.qk_scale_log2 < 0.f ? -1.f : 1.f;
#pragma unroll 1
                for (int b2 = 0; b2 < 2; ++b2) {
                    const int bb = 2 * grp + b2;
                    uint4 raw[4];
                    __half2 top = __half2half2(__ushort_as_half(0));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        raw[k] = row_ok ? src[4 * bb + k] : make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t ws[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __half2 *>(&ws[e])));
                    }
                    // an infinity or NaN in the query: scores of NaN, whatever its codes would be
                    const float2 a2 = __half22float2(top);
                    const float a = fmaxf(a2.x, a2.y);
                    const float sc = a2.x <= 65504.f && a2.y <= 65504.f ? __half2float(__float2half_rn(__fdiv_rn(a, 127.f))) : __int_as_float(0x7fc00000);
                    uint32_t hv[16], lv[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t ws[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&ws[e]));
                            const float2 v = make_float2((float)quant_i8(f.x, sc) * sc * sgn, (float)quant_i8(f.y, sc) * sc * sgn);   // exact: 18 bits
                            hv[4 * k + e] = pack_half2(fminf(fmaxf(v.x, -65504.f), 65504.f), fminf(fmaxf(v.y, -65504.f), 65504.f));   // 127 * 516 is past fp16's range
                            const float2 y = sub2(v, __half22float2(*reinterpret_cast<const __half2 *>(&hv[4 * k + e])));
                            lv[4 * k + e] = pack_half2(y.x, y.y);
                        }
                    }
                    tmem_st16(tQ + lane_base + 16 * bb, hv);
                    tmem_st16(tQ + lane_base + kD / 2 + 16 * bb, lv);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_QR));
                const bool idle_warp = 32 * quarter >= w.R;   // no row here: keep the barriers in step

                const int j1 = j + w.tiles, j0 = j;
                uint32_t a[2][32];
                // This group's half of O, complete with tile t, joins the sums.
                auto join = [&](int t) {
                    float beta = 0.f;
                    const float2 z = *xs;
                    if (t + 1 - j0 > kCFlush<O16>) {   // there are sums
                        beta = z.x == -INFINITY ? 0.f : fast_exp2(z.x - z.y);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float4 y = __ldcg(sums() + k * kCM);
                            uint32_t(&v)[32] = a[k >> 3];
                            v[4 * (k & 7)] = __float_as_uint(y.x);
                            v[4 * (k & 7) + 1] = __float_as_uint(y.y);
                            v[4 * (k & 7) + 2] = __float_as_uint(y.z);
                            v[4 * (k & 7) + 3] = __float_as_uint(y.w);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 64; ++k) a[k >> 5][k & 31] = 0u;
                    }
                    xs->x = z.y;
                    if (!wwait(C::B_PVD + 2 * (t & 1) + 1, (t >> 1) & 1)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[16];
                        tmem_ld16(tO + lane_base + (kD / 2) * grp + 16 * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t *v = &a[q >> 1][16 * (q & 1) + 4 * k];
                            __stcg(sums() + (4 * q + k) * kCM,
                                   make_float4(fmaf(__uint_as_float(v[0]), beta, __uint_as_float(o[4 * k])), fmaf(__uint_as_float(v[1]), beta, __uint_as_float(o[4 * k + 1])),
                                               fmaf(__uint_as_float(v[2]), beta, __uint_as_float(o[4 * k + 2])), fmaf(__uint_as_float(v[3]), beta, __uint_as_float(o[4 * k + 3]))));
                        }
                    }
                    tc_fence_before();
                    return true;
                };
                auto restarts = [&](int t) { return t > j0 && t < j1 && (t - j0) % kCFlush<O16> == 0; };   // O, with P.V(t)
                for (; j < j1; ++j) {
                    if ((j & 1) != grp) continue;   // the other group's tile
                    const uint32_t ph = (j >> 1) & 1;
                    if (idle_warp) {
                        if (!wwait(C::B_SFULL + 2 * grp, ph) || !wwait(C::B_SFULL + 2 * grp + 1, ph)) {
                            lost = true;
                            break;
                        }
                        if (lane == 0) {
                            mbar_arrive(bar(C::B_M + 4 * grp + quarter));
                            mbar_arrive(bar(C::B_PREADY + 2 * grp));
                            mbar_arrive(bar(C::B_PREADY + 2 * grp + 1));
                        }
                        if (restarts(j + 1)) {   // (after P.V(j), as the warps with rows: one arrival each per phase)
                            if (!wwait(C::B_PVD + 2 * grp + 1, ph)) {
                                lost = true;
                                break;
                            }
                            if (lane == 0) mbar_arrive(bar(C::B_OFREE));
                        }
                        continue;
                    }
                    const int x = (w.s0 + j - j0) * kCN;

                    // ---- first pass: the row's maximum, each half as its QK is done ----
                    // (loops are not unrolled beyond a pair of chunks: with every role's code
                    // unrolled the warps waited for instructions)
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        if (!wwait(C::B_SFULL + 2 * grp + i, ph)) {
                            lost = true;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t ts = tSg + kCHalf * i;
                        const int ok = reinterpret_cast<const int *>(smem + C::OREC_OFF)[2 * (j & 3) + i], left = lim - x - kCHalf * i;
                        if (__any_sync(0xffffffffu, ok != 15 || left < kCHalf - 1)) {   // some position is masked: -inf into S
#pragma unroll 1
                            for (int q = 0; q < kCSub; ++q) {
                                uint32_t v[16];
                                tmem_ld16(ts + kWTile * q, v);
                                tmem_wait_ld();
                                const int top = ok >> q & 1 ? left - kWTile * q : -1;
#pragma unroll
                                for (int k = 0; k < 16; ++k) v[k] = k <= top ? v[k] : 0xff800000u;
                                tmem_st16(ts + kWTile * q, v);
                            }
                            tmem_wait_st();
                        }
                        tmem_ld32(ts, a[0]);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t(&v)[32] = a[c];
                            tmem_wait_ld32(v);
                            if (c == 0) tmem_ld32(ts + kCChunk, a[1]);
#pragma unroll
                            for (int k = 0; k < kCChunk; k += 4)
#pragma unroll
                                for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], __uint_as_float(v[k + e]));
                        }
                    }
                    if (lost) break;
                    float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    tmem_ld32(tSg, a[0]);   // the second pass's first chunk
                    mx = mx == -INFINITY ? mx : mx * cs;

                    // ---- the row's zero point after the tile before this one, handed on by the other group ----
                    float mp = -INFINITY;
                    if (j > 0) {
                        if (!wwait(C::B_M + 4 * (grp ^ 1) + quarter, ((j - 1) >> 1) & 1)) {
                            lost = true;
                            break;
                        }
                        if (j > j0) mp = xm[(grp ^ 1) * kCM + row];
                    }
                    const bool need = mx > mp + (kCShift + kCSlack);
                    const float mn = need ? mx - kCShift : mp;
                    xm[grp * kCM + row] = mn;
                    xs->y = restarts(j) ? mp : mn;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_M + 4 * grp + quarter));
                    if (mn != m) {   // raised by either group since this group's last tile
                        l *= m == -INFINITY ? 0.f : fast_exp2(m - mn);
                        m = mn;
                    }
                    if (!restarts(j) && j > j0 && __any_sync(0xffffffffu, need)) {   // O to the new zero point, once P.V(j - 1) is done
                        const float alpha = need ? (mp == -INFINITY ? 0.f : fast_exp2(mp - mn)) : 1.f;
                        if (!wwait(C::B_PVD + 2 * (grp ^ 1) + 1, ((j - 1) >> 1) & 1)) {
                            lost = true;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < kD; c0 += 16) {
                            uint32_t o[16];
                            tmem_ld16(tO + lane_base + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                            tmem_st16(tO + lane_base + c0, o);
                        }
                    }

                    // ---- second pass: P over S, 32 positions at a time ----
                    const float mu = m == -INFINITY ? 0.f : m;
                    const float2 cc = make_float2(cs, cs), nm = make_float2(-mu, -mu);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                    for (int c0 = 0; c0 < kCN; c0 += 2 * kCChunk) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t(&v)[32] = a[c];
                            tmem_wait_ld32(v);
                            if (c == 0 || c0 + 2 * kCChunk < kCN) tmem_ld32(tSg + c0 + kCChunk * (c + 1), a[c ^ 1]);
                            uint32_t hw[16], lw[O16 ? 1 : 16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float2 e = fma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), cc, nm);
                                const float2 pv = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                                sum[k & 1] = add2(sum[k & 1], pv);
                                hw[k] = pack_half2(pv.x, pv.y);
                                if (!O16) {
                                    const float2 y = sub2(pv, __half22float2(*reinterpret_cast<const __half2 *>(&hw[k])));
                                    lw[O16 ? 0 : k] = pack_half2(y.x, y.y);
                                }
                            }
                            tmem_st16(tSg + c0 + kCChunk * c, hw);
                            if constexpr (!O16) tmem_st16(tSg + c0 + kCChunk * c + kCChunk / 2, lw);
                        }
                        tmem_wait_st();   // a half is whole
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0 && !restarts(j)) mbar_arrive(bar(C::B_PREADY + 2 * grp + (c0 ? 1 : 0)));
                    }
                    const float2 s2 = add2(sum[0], sum[1]);
                    l += s2.x + s2.y;
                    // ---- O starts from zero with the P.V of this tile or of the next: its half joins the sums ----
                    if (restarts(j) || restarts(j + 1)) {
                        if (!join(restarts(j) ? j - 1 : j)) {
                            lost = true;
                            break;
                        }
                        __syncwarp();
                        if (lane == 0) {
                            if (restarts(j)) {
                                mbar_arrive(bar(C::B_PREADY + 2 * grp));
                                mbar_arrive(bar(C::B_PREADY + 2 * grp + 1));
                            } else {
                                mbar_arrive(bar(C::B_OFREE));
                            }
                        }
                    }
                }
                // ---- the end of the piece: both groups' sums, and P.V done ----
                if (!lost) {
                    xe[grp * kCM + row] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_END + 4 * grp + quarter));
                    if (!wwait(C::B_END + 4 * (grp ^ 1) + quarter, ends & 1) || !wwait(C::B_PVD + 2 * ((j - 1) & 1) + 1, ((j - 1) >> 1) & 1)) lost = true;
                    ++ends;
                    tc_fence_after();
                    const float2 o = xe[(grp ^ 1) * kCM + row];
                    const float mm = fmaxf(m, o.x);   // O is at the later, higher zero point
                    // without a maximum a sum is 0, or NaN if there were scores
                    l = (m == -INFINITY ? l : l * fast_exp2(m - mm)) + (o.x == -INFINITY ? o.y : o.y * fast_exp2(o.x - mm));
                    m = mm;
                }
            }
            lost = lost || __any_sync(0xffffffffu, *bad != 0);
            // ---- this group's 64 columns of the row out ----
            const bool any = w.tiles > 0 && !(l <= 0.f);
            const float nan = __int_as_float(0x7fc00000);
            float lg;
            asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(l));
            const float f = lost ? nan : any ? 1.0f / l : 0.f;
            const float lse = lost ? nan : any ? (m + lg) * 0.69314718055994531f : -INFINITY;
            const size_t part = ((size_t)blockIdx.x * 2 + max(0, w.slot)) * kCM + row, orow = (size_t)(w.t0 + tok) * p.n_q_heads + head;
            const bool have_o = w.tiles > 0 && !lost, have_sums = have_o && w.tiles > kCFlush<O16>;
            float fs = 0.f;
            if (have_sums) fs = any && xs->x != -INFINITY ? f * fast_exp2(xs->x - m) : 0.f;
#pragma unroll 1
            for (int c0 = (kD / 2) * grp; c0 < (kD / 2) * (grp + 1); c0 += 16) {
                uint32_t o[16];
                if (have_o) {   // warp-uniform
                    tmem_ld16(tO + lane_base + c0, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = 0u;
                }
                if (!row_ok) continue;
                float y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = lost ? nan : any ? __uint_as_float(o[k]) * f : 0.f;
                if (have_sums)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 s = __ldcg(sums() + ((c0 - (kD / 2) * grp) / 4 + k) * kCM);
                        y[4 * k] = fmaf(s.x, fs, y[4 * k]);
                        y[4 * k + 1] = fmaf(s.y, fs, y[4 * k + 1]);
                        y[4 * k + 2] = fmaf(s.z, fs, y[4 * k + 2]);
                        y[4 * k + 3] = fmaf(s.w, fs, y[4 * k + 3]);
                    }
                if (whole && O16) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + orow * kD + c0);
#pragma unroll
                    for (int k = 0; k < 16; k += 8)
                        dst[k / 8] = make_uint4(pack_half2(y[k], y[k + 1]), pack_half2(y[k + 2], y[k + 3]), pack_half2(y[k + 4], y[k + 5]), pack_half2(y[k + 6], y[k + 7]));
                } else {
                    float4 *dst = reinterpret_cast<float4 *>((whole ? static_cast<float *>(p.out) + orow * kD : p.ws_o + part * kD) + c0);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) dst[k / 4] = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                }
            }
            if (row_ok && grp == 0) {
                if (!whole) p.ws_lse[part] = lse;
                else if (p.lse) p.lse[orow] = lse;
            }
            tc_fence_before();
            __syncwarp();
            return true;
        });
        join_roles();
        if (*bad) {   // a wait gave up: every row of this CTA's pieces is NaN, also where no role came to
            const float nan = __int_as_float(0x7fc00000);
            const long long per2 = max((long long)kChunkMinTiles, (line.total + gridDim.x - 1) / gridDim.x), pos2 = per2 * blockIdx.x;
            chunk_pieces(p, line, pos2, min(pos2 + per2, line.total), per2, cuts, [&](const ChunkWalk &w) {
                for (int i = tid; i < w.R * (kD / 4); i += 256) {
                    const int r = i / (kD / 4), d = 4 * (i % (kD / 4));
                    const size_t orow = (size_t)(w.t0 + (w.row0 + r) / w.gsz) * p.n_q_heads + p.grp_q[w.gb + (w.row0 + r) % w.gsz];
                    const size_t part = ((size_t)blockIdx.x * 2 + max(0, w.slot)) * kCM + r;
                    if (w.slot < 0 && O16)
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + orow * kD + d) = make_uint2(0x7fff7fffu, 0x7fff7fffu);
                    else
                        *reinterpret_cast<float4 *>((w.slot < 0 ? static_cast<float *>(p.out) + orow * kD : p.ws_o + part * kD) + d) = make_float4(nan, nan, nan, nan);
                    if (d == 0) {
                        if (w.slot >= 0) p.ws_lse[part] = nan;
                        else if (p.lse) p.lse[orow] = nan;
                    }
                }
                return true;
            });
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kCQk) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int VT>
cudaError_t prepare_chunk_t()
{
    const cudaError_t e = cudaFuncSetAttribute(paged_chunk_kernel<VT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<VT>::SMEM);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(paged_chunk_kernel<VT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<VT>::SMEM);
}

template <int VT, bool LOSE = false>
cudaError_t launch_chunk_t(const PagedAttnParams &p, int out_type, int n_ctas, cudaStream_t s, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_ctas);
    cfg.blockDim = dim3(kChunkThreads);
    cfg.dynamicSmemBytes = ChunkCfg<VT>::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if constexpr (!LOSE)
        if (out_type == KVQ_OUT_F16) return cudaLaunchKernelEx(&cfg, paged_chunk_kernel<VT, true>, p);
    return cudaLaunchKernelEx(&cfg, paged_chunk_kernel<VT, false, LOSE>, p);
}

}  // namespace kvq
