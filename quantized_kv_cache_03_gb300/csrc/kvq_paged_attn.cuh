// kvq_paged_attn.cuh -- attention of a ragged batch over the paged cache: query
// rows in tiles of 8 NT (NT = 1 or 2), mma.sync on the cache's own codes.
//
// Split of the work.  The batch is one line of stages (32 positions of one row
// tile of one kv head): sequence after sequence, kv head after kv head, row
// tile after row tile.  CTA i of the persistent grid takes the i-th equal piece
// of that line, whatever the lengths are, so a batch is one wave without a
// tail.  Every CTA derives its piece from q_start and seq_lens itself (a block
// scan over the sequences), so nothing is planned on the host.  A row tile cut
// by a piece boundary leaves partials (at most two per CTA) for the combine.
//
// A CTA has four warps; warp w takes stages w, w + 4, ... of the piece through
// a private ring filled by bulk copies (a tile record is contiguous: one copy
// per stage, two when pages hold 16 positions).  Nothing but the ring's
// barriers synchronizes the main loop.
//
// Arithmetic per stage (m16n8k16 throughout):
//   scores      K codes enter as 1152 + code; per 32-block an accumulator that
//               starts at -1152 * (sum of the row's codes), so it ends exactly
//               at the integer block dot; score = sum_b I_b * sq_b * sk_b.
//               NT = 2: S = Q K^T, 16 query rows by 8 positions; NT = 1: S^T =
//               K Q^T, 16 positions by 8 query rows (Q as A would leave half of
//               every MMA and fragment empty).
//   O^T += V^T P^T   A = V codes (exact fp16 integers), B = p * d per block.  S
//               (row g, positions 2c, 2c + 1) already has P^T's B layout (k 2c,
//               2c + 1, n = g); S^T is turned by movmatrix.  KVQ_OUT_F32 splits
//               p * d into its upper 11 bits and the rest as fp16 (two MMAs; the
//               rest is rounded to 2^-21 of p * d),
//               KVQ_OUT_F16 rounds it once (2^-11 at most of each term).
// Both outputs sum a stage's P.V from zero and add it in fp32: the MMA's own
// running sum cuts off where fp32 rounds (error against 64 bits on the first batch
// below 4.7e-6 instead of 5e-7).
// Measured: 64 sequences of 1024 to 32768 positions, 4 rows, q8_0 V: 375 us (F16 K
// 508, 0.97 of the bytes' time), 0.91
// of the bytes' time at the measured copy rate; one of 131072 positions, 5 rows,
// q4_0: 48 us (0.67: prologue, merge and combine are a third of it); 16 of 32768,
// 32 rows, fp32 output: 413 us (0.31: 920 instructions per 16 rows and 32
// positions at 46 % issue, two warps per scheduler).
// Softmax in base 2.  A row's reference maximum is raised only when a score
// passes it by more than kSlack = 1, and exponents are taken `shift` above it,
// so p reaches 2^(shift + 1).  That keeps p * d out of fp16's subnormals, where
// the low part loses its bits (d = 1e-5 and p = 1: it has none).  shift follows
// the stage's largest V scale, from the exponent of its bits: p * d_max lies in
// 2^9..2^11 where it may, so 22 bits are kept of terms down to 2^-12 of the
// largest; with d at the top of its range (516 for q8_0, 8188 for q4_0) kShift
// is what still fits fp16.  l carries the same factor, so it cancels.  Shift 24,
// the most, leaves s - m 2^-20 of rounding.
#pragma once

#include "kvq_paged.cuh"
#include "kvq_paged_line.cuh"

namespace kvq {

template <int NT, int VT, int KT>
struct PagedCfg {
    using T = PageTile<VT, KT>;
    static constexpr int WARPS = 4, THREADS = WARPS * 32;
    static constexpr bool F16K = KT == KVQ_K_F16;
    static constexpr int TPS = kStagePos / kWTile;            // tiles per stage
    static constexpr int STAGES = 2;
    static constexpr int STAGE = TPS * T::BYTES, RING = STAGES * STAGE;
    static constexpr int ROWS = 8 * NT;
    static constexpr int KROW = F16K ? 2 * kD : kD;           // bytes of a query row's codes
    static constexpr int Q_OFF = WARPS * RING;
    // int8 K, by block and pair of rows that a lane holds: the accumulators'
    // starts as the MMA takes them, the scales
    static constexpr int PAIRS = ROWS / 2;
    static constexpr int QSEED_OFF = Q_OFF + ROWS * KROW;            // fp32 [kNB][PAIRS][4]
    static constexpr int QS_OFF = QSEED_OFF + kNB * PAIRS * 16;      // fp32 [kNB][PAIRS][2]
    static constexpr int BAR_OFF = QS_OFF + kNB * PAIRS * 8;
    static constexpr int MISC_OFF = BAR_OFF + WARPS * STAGES * 8;
    static constexpr int SMEM = MISC_OFF + 128;
    static constexpr int OROW = kD + 4;
    static constexpr int ML_OFF = WARPS * ROWS * OROW * 4;    // merge: slices, then m, l per warp, then 1/L, lse
    static_assert(ML_OFF + (2 * WARPS + 2) * ROWS * 4 <= WARPS * RING, "the merge reuses the rings");
    static_assert(T::BYTES % 128 == 0 && BAR_OFF % 8 == 0 && QSEED_OFF % 16 == 0, "alignment");
};

// Three CTAs of 8-row tiles per SM, two of 16-row tiles: with a warp more per
// scheduler the accumulators and fragments spill or are loaded too late to
// overlap (131072 positions, 5 rows: 48 us at three, 53 at four, 49 at two;
// 16 sequences of 32 rows, as it was then: 419 us at two, 442 at three).
// LOSE: the test flavour; CTA 0's warp 0 leaves out its copy stage p.lose.
template <int NT, int VT, int KT, bool O16, bool LOSE = false>
__global__ void __launch_bounds__(128, NT == 1 ? 3 : 2) paged_attn_kernel(const __grid_constant__ PagedAttnParams p)
{
    using C = PagedCfg<NT, VT, KT>;
    using T = PageTile<VT, KT>;
    constexpr int W = C::WARPS, S = C::STAGES;
    constexpr float kBias = 1152.0f, kSlack = 1.0f;
    constexpr int kShift = VT == KVQ_V_Q4_0 ? 2 : 5;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LineStart line;
    __shared__ long long tmp[W];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int H = p.pool.n_kv_heads, pshift = p.pool.pshift;
    uint8_t *ring = smem + warp * C::RING;
    const uint32_t ring_s = smem_u32(ring), bar_s = smem_u32(smem + C::BAR_OFF) + warp * S * 8;
    int *bad_flag = reinterpret_cast<int *>(smem + C::MISC_OFF);
    if (tid == 0) *bad_flag = 0;
    if (lane == 0) {
#pragma unroll
        for (int st = 0; st < S; ++st) mbar_init(bar_s + st * 8, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();

    const uint32_t pick = g & 1 ? 0x3232u : 0x1010u;   // NT = 1: the lane's half of a K scale pair, twice
    auto seq_tiles = [&](int n) { return (n * p.gmax + C::ROWS - 1) / C::ROWS; };   // row tiles per kv head
    auto seq_stages = [&](int len) { return max(1, (len + kStagePos - 1) / kStagePos); };
    long long pos, per;
    line_find<C::THREADS>(p, kPagedMinStages, [&](int n, int len, int) { return (long long)H * seq_tiles(n) * seq_stages(len); },
                          &line, tmp, pos, per);
    const long long end = min(pos + per, line.total);
    PagedCut *cuts = p.cuts + (size_t)blockIdx.x * 2;
    if (tid < 2) cuts[tid] = PagedCut{0, 0, 0, 0};
    __syncthreads();
    if (pos >= end) return;

    int b = line.b - 1, t0 = 0, n = 0, L = 0, lim0 = 0, n_st = 0, n_rt = 0, h = 0, rt = 0, s0 = 0;
    bool fresh = true;
    int done = 0;   // stages this warp has taken since the kernel began: ring slot and phase
    const bool loser = LOSE && blockIdx.x == 0 && warp == 0;
    for (bool first = true; pos < end; first = false) {
        if (fresh) {   // next sequence of this launch
            do {
                ++b;
                seq_shape(p, b, t0, n, L, lim0);
            } while (!seq_mine(p, n));
            n_st = seq_stages(L);
            n_rt = seq_tiles(n);
            h = rt = s0 = 0;
            if (first) {
                const long long u = line.off / n_st;
                s0 = (int)(line.off - u * n_st);
                rt = (int)(u % n_rt);
                h = (int)(u / n_rt);
            }
            fresh = false;
        }
        const int s1 = (int)min((long long)n_st, s0 + (end - pos));
        const int gb = p.grp_begin[h], gsz = p.grp_begin[h + 1] - gb;
        const int row0 = rt * C::ROWS, R = min(C::ROWS, n * gsz - row0);   // row r: token (row0 + r) / gsz of the sequence
        const bool whole = s0 == 0 && s1 == n_st;
        const int slot = s0 == 0 ? 1 : 0;
        if (R > 0) {
            if (!whole && tid == 0) {
                const long long x0 = pos - s0, c0 = x0 / per;   // CTA that begins the row tile
                cuts[slot] = PagedCut{b, h | rt << 8, (int)c0, (int)((x0 + n_st - 1) / per - c0 + 1)};
            }
            // positions the tile's last and first rows see end at lim_hi, lim_lo
            const int lim_hi = p.causal ? lim0 + (row0 + R - 1) / gsz : L - 1;
            const int lim_lo = p.causal ? lim0 + row0 / gsz : L - 1;
            const int sv = min(s1, (lim_hi + kStagePos) / kStagePos);       // stages past sv show nothing (lim_hi >= -kStagePos)
            const int nj = lim_hi < 0 ? 0 : max(0, (sv - s0 - warp + W - 1) / W);   // this warp's stages

            // ---- page ids, 32 stages ahead per load ----
            const int *bt = p.block_table + (size_t)b * p.table_stride;
            int pg0 = -1, pg1 = -1, okm = 0, issued = 0;
            auto fetch = [&](int j) {   // lane l: stage j + l
                const int x = (s0 + warp + W * (j + lane)) * kStagePos;
                pg0 = pg1 = -1;
                if (j + lane < nj) {
                    pg0 = bt[x >> pshift];
                    if (pshift == 4 && x + 16 < L) pg1 = bt[(x >> 4) + 1];
                }
            };
            auto issue = [&]() {
                if ((issued & 31) == 0) fetch(issued);
                const int sl = (done + issued) % S;   // `done` counts finished pieces' stages only
                const int a0 = __shfl_sync(0xffffffffu, pg0, issued & 31);
                const int x = (s0 + warp + W * issued) * kStagePos;
                const int tile = (x & ((1 << pshift) - 1)) >> 4;
                const bool v0 = a0 >= 0 && a0 < p.pool.n_pages;
                const uint32_t dst = ring_s + sl * C::STAGE, bw = bar_s + sl * 8;
                const bool drop = LOSE && loser && done + issued == p.lose;
                int ok;
                if (pshift == 4) {
                    const int a1 = __shfl_sync(0xffffffffu, pg1, issued & 31);
                    const bool v1 = a1 >= 0 && a1 < p.pool.n_pages;
                    ok = (v0 ? 1 : 0) | (v1 ? 2 : 0);
                    mbar_arrive_expect_tx_w(bw, ((v0 ? 1 : 0) + (v1 ? 1 : 0)) * T::BYTES);
                    if (v0 && !drop) bulk_g2s_w(dst, tile_of(p.pool, a0, h, 0, T::BYTES), T::BYTES, bw);
                    if (v1 && !drop) bulk_g2s_w(dst + T::BYTES, tile_of(p.pool, a1, h, 0, T::BYTES), T::BYTES, bw);
                } else {
                    ok = v0 ? 3 : 0;
                    mbar_arrive_expect_tx_w(bw, v0 ? C::STAGE : 0);
                    if (v0 && !drop) bulk_g2s_w(dst, tile_of(p.pool, a0, h, tile, T::BYTES), C::STAGE, bw);
                }
                okm = (okm & ~(3 << (2 * sl))) | ok << (2 * sl);
                ++issued;
            };
            // a warp that lost a copy issues nothing more (its results are poisoned)
            const int nj_live = *bad_flag ? 0 : nj;
#pragma unroll
            for (int k = 0; k < S; ++k)
                if (issued < nj_live) issue();

            // ---- query rows -> fragments ----
            uint32_t qa[8][2 * NT];            // [k16 step][row g: k 2c.., k 2c + 8..; row g + 8 likewise]
            // the two rows whose scores the lane holds: 2c, 2c + 1 (NT = 1), g, g + 8 (NT = 2)
            const int lrow[2] = {NT == 1 ? 2 * c : g, NT == 1 ? 2 * c + 1 : g + 8};
            // int8 K: read again for each stage, the registers hold enough
            float4 *qseed = reinterpret_cast<float4 *>(smem + C::QSEED_OFF);
            float2 *qs = reinterpret_cast<float2 *>(smem + C::QS_OFF);
            const int pair = NT == 1 ? c : g;
            {
                uint32_t *qw = reinterpret_cast<uint32_t *>(smem + C::Q_OFF);
#pragma unroll
                for (int k = 0; k < C::ROWS / W; ++k) {
                    const int r = warp + W * k;
                    uint2 raw = make_uint2(0u, 0u);
                    if (r < R) {
                        const size_t t = t0 + (row0 + r) / gsz;
                        raw = *reinterpret_cast<const uint2 *>(p.q + t * p.q_stride + (size_t)p.grp_q[gb + (row0 + r) % gsz] * kD + 4 * lane);
                    }
                    // a row with an infinity or NaN gets scores of NaN, whatever its codes would be
                    const __half2 top = __hmax2_nan(__habs2(*reinterpret_cast<const __half2 *>(&raw.x)), __habs2(*reinterpret_cast<const __half2 *>(&raw.y)));
                    const bool wild = __any_sync(0xffffffffu, !__hble2(top, __half2half2(__ushort_as_half(0x7bff))));
                    if (C::F16K) {
                        *reinterpret_cast<uint2 *>(qw + r * (kD / 2) + 2 * lane) = wild ? make_uint2(0x7fff7fffu, 0x7fff7fffu) : raw;
                        continue;
                    }
                    const float2 lo = half2_of(raw.x), hi = half2_of(raw.y);
                    const float xv[4] = {lo.x, lo.y, hi.x, hi.y};
                    uint16_t s16;
                    const uint32_t word = quant_row_i8(xv, s16);
                    int sum = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum += (int)(int8_t)(word >> (8 * e));
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    qw[r * (kD / 4) + lane] = word;
                    if ((lane & 7) == 0) {
                        const int x = (lane >> 3) * C::PAIRS + (NT == 1 ? r >> 1 : r & 7), e = NT == 1 ? r & 1 : r >> 3;
                        float *sd = reinterpret_cast<float *>(qseed + x);
                        reinterpret_cast<float *>(qs + x)[e] = wild ? __int_as_float(0x7fc00000) : __half2float(__ushort_as_half(s16)) * p.qk_scale_log2;
                        sd[NT == 1 ? e : 2 * e] = sd[NT == 1 ? e + 2 : 2 * e + 1] = -kBias * (float)sum;
                    }
                }
                __syncthreads();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int r = g + 8 * nt;
                    if (C::F16K) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            qa[ks][2 * nt] = qw[r * (kD / 2) + 8 * ks + c];
                            qa[ks][2 * nt + 1] = qw[r * (kD / 2) + 8 * ks + c + 4];
                        }
                    } else {
#pragma unroll
                        for (int bb = 0; bb < kNB; ++bb) {
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk) {
                                const uint32_t w = qw[r * (kD / 4) + 8 * bb + 2 * c + kk];
                                qa[2 * bb + kk][2 * nt] = code_pair(w, 0);
                                qa[2 * bb + kk][2 * nt + 1] = code_pair(w, 2);
                            }
                        }
                    }
                }
            }
            float m[2], l[2], mu[2];
            int lim[2];
            float acc[8][NT][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                lim[e] = lrow[e] < R ? (p.causal ? lim0 + (row0 + lrow[e]) / gsz : L - 1) : -1;
                m[e] = -INFINITY;
                mu[e] = l[e] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[mt][nt][k] = 0.f;

            int lost = -1;   // the stage whose wait gave up
#pragma unroll 1
            for (int j = 0; j < nj_live; ++j) {
                const int sl = (done + j) % S;
                const uint32_t spins = LOSE && loser && done + j == p.lose ? kLostCopySpins : kMbarSpins;
                if (!__all_sync(0xffffffffu, mbar_wait(bar_s + sl * 8, ((done + j) / S) & 1, spins))) {
                    lost = j;
                    break;
                }
                uint8_t *stg = ring + sl * C::STAGE;
                const int x = (s0 + warp + W * j) * kStagePos, ok = (okm >> (2 * sl)) & 3;
                const bool full = ok == 3 && x + kStagePos - 1 <= lim_lo;   // every row sees the whole stage
                {
                    // the lane's four of the stage's V scales
                    uint2 *d4 = reinterpret_cast<uint2 *>(stg + (lane >> 4) * T::BYTES + T::VS_OFF + 8 * (lane & 15));
                    uint2 dv = *d4;
                    if (!full) {
                        // V scales of positions that no row sees may hold anything: p is 0 there, make d so too
                        const int t = lane >> 4, q1 = x + 16 * t + 2 * ((lane & 15) >> 1);
                        const uint32_t keep = !((ok >> t) & 1) ? 0u : (q1 <= lim_hi ? 0xffffu : 0u) | (q1 + 1 <= lim_hi ? 0xffff0000u : 0u);
                        dv = make_uint2(dv.x & keep, dv.y & keep);
                        *d4 = dv;
                        __syncwarp();
                    }
                    // d_max < 2^(e - 14), e its exponent bits: 2^shift * d_max in 2^9..2^10
                    const uint32_t dm = __vmaxu2(dv.x, dv.y);
                    const int de = (int)(__reduce_max_sync(0xffffffffu, max(dm & 0xffffu, dm >> 16)) >> 10);
                    const float shift = (float)max(kShift, 24 - de);
                    // scores of 8-position group i (of four): NT = 1 position 8i + g, rows (2c, 2c + 1);
                    // NT = 2 positions (8i + 2c, + 1), [row g, row g + 8]
                    float2 s[NT][4];
                    if constexpr (C::F16K) {
#pragma unroll
                        for (int t = 0; t < C::TPS; ++t) {
                            float d[2][4] = {};
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks) {
                                const uint4 k4 = *reinterpret_cast<const uint4 *>(stg + t * T::BYTES + ks * 512 + lane * 16);
                                if constexpr (NT == 1) {
                                    const uint32_t a[4] = {k4.x, k4.y, k4.z, k4.w};
                                    mma_f16_16816(d[0], a, qa[ks][0], qa[ks][1]);
                                } else {
                                    const uint32_t a[4] = {qa[ks][0], qa[ks][2 * NT - 2], qa[ks][1], qa[ks][2 * NT - 1]};
                                    mma_f16_16816(d[0], a, k4.x, k4.z);
                                    mma_f16_16816(d[1], a, k4.y, k4.w);
                                }
                            }
                            const float2 sc = make_float2(p.qk_scale_log2, p.qk_scale_log2);
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if constexpr (NT == 1) {
                                    s[0][2 * t + i] = mul2(make_float2(d[0][2 * i], d[0][2 * i + 1]), sc);
                                } else {
                                    s[0][2 * t + i] = mul2(make_float2(d[i][0], d[i][1]), sc);
                                    s[NT - 1][2 * t + i] = mul2(make_float2(d[i][2], d[i][3]), sc);
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int hb = 0; hb < 2; ++hb) {   // blocks 2hb, 2hb + 1
                            uint4 kk[C::TPS][2];
                            uint2 sk[C::TPS][2];           // NT = 1: the scale pairs of positions 2 (g/2), + 1; NT = 2: of 2c, 2c + 1
#pragma unroll
                            for (int t = 0; t < C::TPS; ++t)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint8_t *tk = stg + t * T::BYTES;
                                    kk[t][i] = *reinterpret_cast<const uint4 *>(tk + (2 * i + hb) * 512 + lane * 16);
                                    sk[t][i] = *reinterpret_cast<const uint2 *>(tk + T::KS_OFF + (4 * i + (NT == 1 ? g >> 1 : c)) * 16 + 8 * hb);
                                }
#pragma unroll
                            for (int bb = 2 * hb; bb < 2 * hb + 2; ++bb) {
                                const uint4 seed = *reinterpret_cast<const uint4 *>(qseed + bb * C::PAIRS + pair);
                                const float2 sq = qs[bb * C::PAIRS + pair];
#pragma unroll
                                for (int t = 0; t < C::TPS; ++t) {
                                    uint32_t lo[2][2], hi[2][2];   // [position group][k16 step]: K bytes 0, 1 and 2, 3 as 1152 + code
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        const uint4 &kw = kk[t][i];
                                        const uint32_t w0 = (bb & 1) ? kw.z : kw.x, w1 = (bb & 1) ? kw.w : kw.y;
                                        lo[i][0] = __byte_perm(w0, 0x64646464u, 0x4140);
                                        hi[i][0] = __byte_perm(w0, 0x64646464u, 0x4342);
                                        lo[i][1] = __byte_perm(w1, 0x64646464u, 0x4140);
                                        hi[i][1] = __byte_perm(w1, 0x64646464u, 0x4342);
                                    }
                                    if constexpr (NT == 1) {   // S^T = K Q^T: rows are the 16 positions
                                        float d[4];
                                        const uint32_t a0[4] = {lo[0][0], lo[1][0], hi[0][0], hi[1][0]}, a1[4] = {lo[0][1], lo[1][1], hi[0][1], hi[1][1]};
                                        mma_f16_16816_c4(d, a0, qa[2 * bb][0], qa[2 * bb][1], seed);
                                        mma_f16_16816(d, a1, qa[2 * bb + 1][0], qa[2 * bb + 1][1]);
#pragma unroll
                                        for (int i = 0; i < 2; ++i) {
                                            const uint32_t sw = (bb & 1) ? sk[t][i].y : sk[t][i].x;
                                            const float f = half2_of(__byte_perm(sw, sw, pick)).x;
                                            const float2 v = mul2(make_float2(d[2 * i], d[2 * i + 1]), sq), s2 = make_float2(f, f);
                                            s[0][2 * t + i] = bb == 0 ? mul2(v, s2) : fma2(v, s2, s[0][2 * t + i]);
                                        }
                                    } else {                   // S = Q K^T: rows are the query rows
#pragma unroll
                                        for (int i = 0; i < 2; ++i) {
                                            float d[4];
                                            const uint32_t a0[4] = {qa[2 * bb][0], qa[2 * bb][2 * NT - 2], qa[2 * bb][1], qa[2 * bb][2 * NT - 1]};
                                            const uint32_t a1[4] = {qa[2 * bb + 1][0], qa[2 * bb + 1][2 * NT - 2], qa[2 * bb + 1][1], qa[2 * bb + 1][2 * NT - 1]};
                                            mma_f16_16816_c4(d, a0, lo[i][0], hi[i][0], seed);
                                            mma_f16_16816(d, a1, lo[i][1], hi[i][1]);
                                            const float2 s2 = half2_of((bb & 1) ? sk[t][i].y : sk[t][i].x);
#pragma unroll
                                            for (int nt = 0; nt < NT; ++nt) {
                                                const float q1 = nt == 0 ? sq.x : sq.y;
                                                const float2 v = mul2(make_float2(d[2 * nt], d[2 * nt + 1]), make_float2(q1, q1));
                                                s[nt][2 * t + i] = bb == 0 ? mul2(v, s2) : fma2(v, s2, s[nt][2 * t + i]);
                                            }
                                        }
                                    }
                                }
                            }
                        }
                    }
                    if (!full) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int q0 = x + 8 * i + (NT == 1 ? g : 2 * c);
                            const bool live = (ok >> (i >> 1)) & 1;
                            if constexpr (NT == 1) {
                                s[0][i].x = live && q0 <= lim[0] ? s[0][i].x : -INFINITY;
                                s[0][i].y = live && q0 <= lim[1] ? s[0][i].y : -INFINITY;
                            } else {
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    s[nt][i].x = live && q0 <= lim[nt] ? s[nt][i].x : -INFINITY;
                                    s[nt][i].y = live && q0 + 1 <= lim[nt] ? s[nt][i].y : -INFINITY;
                                }
                            }
                        }
                    }
                    // ---- softmax: a row's scores sit in the eight lanes of one c (NT = 1) or the four of one g ----
                    float mx[2];
                    if constexpr (NT == 1) {
                        mx[0] = fmaxf(fmaxf(s[0][0].x, s[0][1].x), fmaxf(s[0][2].x, s[0][3].x));
                        mx[1] = fmaxf(fmaxf(s[0][0].y, s[0][1].y), fmaxf(s[0][2].y, s[0][3].y));
                    } else {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mx[nt] = fmaxf(fmaxf(fmaxf(s[nt][0].x, s[nt][0].y), fmaxf(s[nt][1].x, s[nt][1].y)),
                                           fmaxf(fmaxf(s[nt][2].x, s[nt][2].y), fmaxf(s[nt][3].x, s[nt][3].y)));
                    }
                    const bool need = mx[0] > m[0] + (shift + kSlack) || mx[1] > m[1] + (shift + kSlack);
                    if (__any_sync(0xffffffffu, need)) {
                        float al[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float v = mx[e];
                            if constexpr (NT == 1) {
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                            } else {
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                            }
                            v = fmaxf(m[e], v - shift);   // m: the exponents' zero
                            al[e] = v == -INFINITY ? 1.f : fast_exp2(m[e] - v);
                            l[e] *= al[e];
                            m[e] = v;
                            mu[e] = v == -INFINITY ? 0.f : v;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            // the accumulator's columns are rows 8 nt + 2c, + 1; with NT = 2 their factors sit in lanes 8c, 8c + 4
                            float2 a2 = make_float2(al[0], al[1]);
                            if constexpr (NT == 2) a2 = make_float2(__shfl_sync(0xffffffffu, al[nt], 8 * c), __shfl_sync(0xffffffffu, al[nt], 8 * c + 4));
#pragma unroll
                            for (int mt = 0; mt < 8; ++mt) {
                                const float2 lo = mul2(make_float2(acc[mt][nt][0], acc[mt][nt][1]), a2);
                                const float2 hi = mul2(make_float2(acc[mt][nt][2], acc[mt][nt][3]), a2);
                                acc[mt][nt][0] = lo.x; acc[mt][nt][1] = lo.y;
                                acc[mt][nt][2] = hi.x; acc[mt][nt][3] = hi.y;
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float2 m2 = NT == 1 ? make_float2(mu[0], mu[1]) : make_float2(mu[nt], mu[nt]);
                        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 e = sub2(s[nt][i], m2);
                            s[nt][i] = make_float2(fast_exp2(e.x), fast_exp2(e.y));
                            sum = add2(sum, s[nt][i]);
                        }
                        if constexpr (NT == 1) {
                            l[0] += sum.x;
                            l[1] += sum.y;
                        } else {
                            l[nt] += sum.x + sum.y;
                        }
                    }
                    if constexpr (NT == 1) {   // (position, row) to (row, position): each fp32's halves turned as 8x8 matrices
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a = __float_as_uint(s[0][i].x), b2 = __float_as_uint(s[0][i].y);
                            const uint32_t lo = movmatrix_t(__byte_perm(a, b2, 0x5410)), hi = movmatrix_t(__byte_perm(a, b2, 0x7632));
                            s[0][i] = make_float2(__uint_as_float(__byte_perm(lo, hi, 0x5410)), __uint_as_float(__byte_perm(lo, hi, 0x7632)));
                        }
                    }
                    // ---- O^T += V^T P^T, block by block ----
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {   // blocks 2hb, 2hb + 1
                        uint4 vv[C::TPS][2];           // their V codes: q4 in x, y only
                        uint2 sv[C::TPS][2];
#pragma unroll
                        for (int t = 0; t < C::TPS; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint8_t *tv = stg + t * T::BYTES + T::V_OFF, *ts = stg + t * T::BYTES + T::VS_OFF;
                                if (VT == KVQ_V_Q4_0) {
                                    const uint2 w = *reinterpret_cast<const uint2 *>(tv + i * 512 + lane * 16 + 8 * hb);
                                    vv[t][i] = make_uint4(w.x, w.y, 0u, 0u);
                                } else {
                                    vv[t][i] = *reinterpret_cast<const uint4 *>(tv + (2 * i + hb) * 512 + lane * 16);
                                }
                                sv[t][i] = *reinterpret_cast<const uint2 *>(ts + (4 * i + c) * 16 + 8 * hb);
                            }
#pragma unroll
                      for (int bb = 2 * hb; bb < 2 * hb + 2; ++bb) {
                        // fp32 output: the stage's part is summed from zero and then added, so that the MMA's
                        // truncating additions do not run over the whole sum (twice the plain form's error)
                        float part[2][NT][4];
#pragma unroll
                        for (int t = 0; t < C::TPS; ++t) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t r[2][2];
                                const uint4 &v = vv[t][i];
                                if (VT == KVQ_V_Q4_0) v_codes<VT>((bb & 1) ? v.y : v.x, 0u, r);
                                else v_codes<VT>((bb & 1) ? v.z : v.x, (bb & 1) ? v.w : v.y, r);
                                a[0][2 * i] = r[0][0];
                                a[0][2 * i + 1] = r[0][1];
                                a[1][2 * i] = r[1][0];
                                a[1][2 * i + 1] = r[1][1];
                            }
                            float2 d2[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t dw = (bb & 1) ? sv[t][i].y : sv[t][i].x;
                                d2[i] = half2_of(dw);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint32_t hi[2], lo[2];
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float2 xv = mul2(s[nt][2 * t + i], d2[i]);
                                    if (O16) {
                                        hi[i] = pack_half2(xv.x, xv.y);
                                    } else {   // the upper 11 bits by a mask (the ALU has room: 419 -> 407 us), and what they leave out
                                        const float2 h = make_float2(__uint_as_float(__float_as_uint(xv.x) & 0xffffe000u), __uint_as_float(__float_as_uint(xv.y) & 0xffffe000u));
                                        const float2 y = sub2(xv, h);
                                        hi[i] = pack_half2(h.x, h.y);
                                        lo[i] = pack_half2(y.x, y.y);
                                    }
                                }
#pragma unroll
                                for (int h2 = 0; h2 < 2; ++h2) {
                                    if (t == 0) mma_f16_16816_c4(part[h2][nt], a[h2], hi[0], hi[1], make_uint4(0u, 0u, 0u, 0u));
                                    else mma_f16_16816(part[h2][nt], a[h2], hi[0], hi[1]);
                                    if (!O16) mma_f16_16816(part[h2][nt], a[h2], lo[0], lo[1]);
                                }
                            }
                        }
#pragma unroll
                            for (int h2 = 0; h2 < 2; ++h2)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float(&o)[4] = acc[2 * bb + h2][nt];
                                    const float2 u0 = add2(make_float2(o[0], o[1]), make_float2(part[h2][nt][0], part[h2][nt][1]));
                                    const float2 u1 = add2(make_float2(o[2], o[3]), make_float2(part[h2][nt][2], part[h2][nt][3]));
                                    o[0] = u0.x; o[1] = u0.y; o[2] = u1.x; o[3] = u1.y;
                                }
                      }
                    }
                }
                __syncwarp();   // every lane has read the slot
                if (issued < nj_live) {
                    fence_proxy_async_smem();
                    issue();
                }
            }
            if (lost >= 0) {   // wait (bounded) for the copies in flight, then poison this piece and the later ones
                for (int k = lost; k < issued; ++k)
                    if (!(LOSE && loser && done + k == p.lose)) mbar_wait(bar_s + ((done + k) % S) * 8, ((done + k) / S) & 1);
                if (lane == 0) {
                    atomicOr(bad_flag, 1);
                    atomicAdd(p.timeouts, 1u);
                }
            }
            done += nj_live;

            // ---- merge the warps in a fixed order and write ----
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], NT == 1 ? 4 : 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], NT == 1 ? 8 : 2);
                if (NT == 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
            }
            __syncthreads();   // every warp is done with its ring
            float *sm_o = reinterpret_cast<float *>(smem), *sm_m = reinterpret_cast<float *>(smem + C::ML_OFF);
            float *sm_l = sm_m + W * C::ROWS, *sm_inv = sm_l + W * C::ROWS, *sm_lse = sm_inv + C::ROWS;
            if (NT == 1 ? g == 0 : c == 0)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sm_m[warp * C::ROWS + lrow[e]] = m[e];
                    sm_l[warp * C::ROWS + lrow[e]] = l[e];
                }
            __syncthreads();
            if (tid < R) {
                float M = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) M = fmaxf(M, sm_m[w * C::ROWS + tid]);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float mw = sm_m[w * C::ROWS + tid];
                    const float lw = sm_l[w * C::ROWS + tid];   // without a maximum: 0, or NaN if there were scores
                    sum += mw == -INFINITY ? lw : lw * fast_exp2(mw - M);
                }
                float lg;
                asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(sum));
                const bool any = !(sum <= 0.f);
                sm_inv[tid] = any ? __fdividef(1.f, sum) : 0.f;
                sm_lse[tid] = any ? (M + lg) * 0.69314718055994531f : -INFINITY;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * nt + 2 * c + e;   // the accumulator's column
                    float M = -INFINITY;
#pragma unroll
                    for (int w = 0; w < W; ++w) M = fmaxf(M, sm_m[w * C::ROWS + r]);
                    const float mw = sm_m[warp * C::ROWS + r], f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
#pragma unroll
                    for (int mt = 0; mt < 8; ++mt)
                        *reinterpret_cast<float2 *>(&sm_o[(warp * C::ROWS + r) * C::OROW + v_dim<VT>(mt, g)]) =
                            make_float2(acc[mt][nt][e] * f, acc[mt][nt][2 + e] * f);
                }
            __syncthreads();
            const bool poisoned = *bad_flag != 0;
            for (int i4 = tid; i4 < R * (kD / 4); i4 += C::THREADS) {
                const int r = i4 / (kD / 4), d = (i4 % (kD / 4)) * 4;
                float4 o = *reinterpret_cast<const float4 *>(&sm_o[r * C::OROW + d]);
#pragma unroll
                for (int w = 1; w < W; ++w) {
                    const float4 q = *reinterpret_cast<const float4 *>(&sm_o[(w * C::ROWS + r) * C::OROW + d]);
                    o.x += q.x; o.y += q.y; o.z += q.z; o.w += q.w;
                }
                const float inv = sm_inv[r];
                float ls = sm_lse[r];
                o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
                if (poisoned) o.x = o.y = o.z = o.w = ls = __int_as_float(0x7fc00000);
                if (whole) {
                    const size_t row = (size_t)(t0 + (row0 + r) / gsz) * p.n_q_heads + p.grp_q[gb + (row0 + r) % gsz];
                    if (O16)
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row * kD + d) = make_uint2(pack_half2(o.x, o.y), pack_half2(o.z, o.w));
                    else
                        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + row * kD + d) = o;
                    if (d == 0 && p.lse) p.lse[row] = ls;
                } else {
                    const size_t at = ((size_t)blockIdx.x * 2 + slot) * C::ROWS + r;
                    *reinterpret_cast<float4 *>(p.ws_o + at * kD + d) = o;
                    if (d == 0) p.ws_lse[at] = ls;
                }
            }
            fence_proxy_async_smem();   // these accesses before the copies of the next piece
            __syncthreads();            // the rings are free again
        }
        pos += s1 - s0;
        s0 = 0;
        if (++rt == n_rt) {
            rt = 0;
            if (++h == H) fresh = true;
        }
    }
}

template <int NT, int VT, int KT, bool O16>
cudaError_t prepare_paged_t(int *ctas)
{
    using C = PagedCfg<NT, VT, KT>;
    const void *fn = (const void *)paged_attn_kernel<NT, VT, KT, O16>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, fn, C::THREADS, C::SMEM);
}

// pdl only for grids of one CTA per SM at most: beside the last blocks of the
// launch in front, the three or four CTAs that fill an SM's shared memory can
// leave a hole that the last of them does not fit, and it then starts only when
// another has finished (64 sequences, 456 CTAs: 370 us or up to 480 us).
template <int NT, int VT, int KT, bool O16, bool LOSE = false>
cudaError_t launch_paged_t(const PagedAttnParams &p, int n_ctas, cudaStream_t s, bool pdl)
{
    using C = PagedCfg<NT, VT, KT>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attn_kernel<NT, VT, KT, O16, LOSE>, p);
}

#define KVQ_PAGED_PICK(FN, VT, nt, k_type, out_type, ...)                                                              \
    ((k_type) == KVQ_K_F16                                                                                             \
         ? ((nt) == 1 ? ((out_type) == KVQ_OUT_F16 ? FN<1, VT, KVQ_K_F16, true>(__VA_ARGS__) : FN<1, VT, KVQ_K_F16, false>(__VA_ARGS__))  \
                      : ((out_type) == KVQ_OUT_F16 ? FN<2, VT, KVQ_K_F16, true>(__VA_ARGS__) : FN<2, VT, KVQ_K_F16, false>(__VA_ARGS__))) \
         : ((nt) == 1 ? ((out_type) == KVQ_OUT_F16 ? FN<1, VT, KVQ_K_I8, true>(__VA_ARGS__) : FN<1, VT, KVQ_K_I8, false>(__VA_ARGS__))    \
                      : ((out_type) == KVQ_OUT_F16 ? FN<2, VT, KVQ_K_I8, true>(__VA_ARGS__) : FN<2, VT, KVQ_K_I8, false>(__VA_ARGS__))))

#define KVQ_DEFINE_PAGED_ENTRY(SUFFIX, VT)                                                                           \
    cudaError_t prepare_paged_##SUFFIX(int nt, int k_type, int out_type, int *ctas)                                  \
    {                                                                                                                \
        return KVQ_PAGED_PICK(prepare_paged_t, VT, nt, k_type, out_type, ctas);                                      \
    }                                                                                                                \
    cudaError_t launch_paged_##SUFFIX(const PagedAttnParams &p, int nt, int k_type, int out_type, int n_ctas,        \
                                      cudaStream_t s, bool pdl)                                                      \
    {                                                                                                                \
        return KVQ_PAGED_PICK(launch_paged_t, VT, nt, k_type, out_type, p, n_ctas, s, pdl);                          \
    }

}  // namespace kvq
