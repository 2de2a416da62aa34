// Attention over a 4-bit prefix cache on tcgen05 tensor cores (BF16 mode).
//
// The codes become bf16 in shared memory, next to the MMAs that read them, so
// only 4.5 bits an element cross HBM and L2. The values of the format are exact
// in bf16: S = Q K^T and O = P V are the products a bf16 cache holding the same
// values would give. The weights P are rounded to bf16 (2^-8 of each at most), because
// both operands of a product have one type; sums, maxima and outputs are fp32.
//
// Work is cut into steps of one 128-key tile of one unit (item, head, query
// tile); the steps of all units, laid end to end, are shared out evenly over one
// CTA an SM. A CTA walks its segments (runs of steps of one unit); a unit that
// lies in one CTA is finished there, one that was cut leaves a normalised fp32
// partial result with its log2-sum-exp for k_kv4_join. Units of the same head
// are neighbours, so CTAs that run together read the same K/V from L2.
//   Two arrangements of the two softmax halves A and B (each with its own S and O
// accumulators in TMEM):
//   * more than 128 query rows: a unit is 256 rows, half A the first 128, half B
//     the others. Each K/V tile serves both, so it is expanded once for 256 rows.
//   * up to 128 rows: both halves hold the same rows and take the first and the
//     second half of the segment's key tiles (the epilogue merges them), because
//     a single half leaves the tensor pipe idle while its softmax runs.
//   warps 0..3, 4..7 : softmax of half A and B, one thread per query row
//   warps 8..11      : K/V producers. Prefix tiles: codes and scales from a
//                      staging ring, expanded to bf16 in the 128-byte-swizzled
//                      operand layout. Tail tiles: TMA loads into the same ring.
//   warp 12          : TMEM allocator + UMMA issuer
//   warp 13, 14      : bulk copies of codes and scales into the staging ring; Q loads
// Bound by the expansion (four warps, 860 cycles a tile alone, twice that beside the
// softmax) and the chain of the softmax: 145 us for 256 rows over P 33792, 32 heads of
// 128 (980 TFLOP/s), 69 us for 512 rows over 4608 + 512 keys; two producer warps instead
// of four (and 168 registers for all) 297 us for the former.
// Registers: 512 threads launched with 128 each; the softmax warpgroups (128
// scores a row in registers) take 192 each, the producers 72, the last 56
// (192 + 192 + 72 + 56 = 4 x 128).
// Expanding costs two instructions an element: nibbles i and i + 4 of a code word
// are masked into the mantissas of a bf16 pair as 16 + nibble (0x4180 | nibble <<
// 3), one fma.bf16x2 forms (16 + nibble) s - 24 s = (nibble - 8) s without
// rounding (24 s has at most 7 bits), and byte permutes restore the order of dims.
#pragma once
#include "qi21_attn_tc.cuh"
#include "qi21_kv4.cuh"

namespace qi21 {

template <int DH>
struct Kv4AttnCfg {
    static constexpr int BQ = 128, BK = 128, BOXES = DH / 64;
    static constexpr int G = DH / KV4_GROUP;
    static constexpr int Q_BYTES = BQ * DH * 2, KV_BYTES = BK * DH * 2;
    static constexpr int CODE_BYTES = BK * DH / 2, SCALE_BYTES = BK * G * 2;
    static constexpr int STAGE_BYTES = CODE_BYTES + SCALE_BYTES;
    static constexpr int NS = 3;                              // staging ring (K and V tiles alternate)
    static constexpr int OFF_Q = 0;                           // two halves
    static constexpr int OFF_K = OFF_Q + 2 * Q_BYTES;         // 2 stages
    static constexpr int OFF_V = OFF_K + 2 * KV_BYTES;        // 2 stages
    static constexpr int OFF_ST = OFF_V + 2 * KV_BYTES;
    static constexpr int OFF_BAR = OFF_ST + NS * STAGE_BYTES;
    static constexpr int OFF_STATS = OFF_BAR + 256;           // [2 parities][2 halves][m, l][128] floats
    static constexpr size_t SMEM = (size_t)OFF_STATS + 2 * 2 * 2 * BQ * 4;
    static constexpr int THREADS = 512;
};

// First step of a CTA's range (kv4_plan() fills Kv4Work).
__host__ __device__ __forceinline__ int64_t kv4_work_begin(const Kv4Work &w, int cta) {
    const int64_t n = w.whole ? w.units : (int64_t)w.units * w.tiles, p = n * cta;
    const int64_t at = (p >> 32) == 0 ? (int64_t)((uint32_t)p / (uint32_t)w.grid) : p / w.grid;   // 32 bits are cheaper
    return w.whole ? at * w.tiles : at;
}

struct Kv4TcArgs {
    Kv4AttnArgs a;
    Kv4Work w;
    float *part_l;               // [2 grid][slot_rows]
    float *part_o;               // [2 grid][slot_rows][DH]
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int R>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Expand one 128-row tile of codes (rows of DH/2 bytes) into the swizzled operand
// buffer at dst (boxes of 64 dims, rows of 128 bytes) with W warps; rows from n_rows
// on become zeros (their scale is taken as 0). A quarter warp covers four rows and
// two groups: its eight 16-byte stores fall into eight different chunks of the
// swizzle.
template <int DH, int W>
__device__ __forceinline__ void kv4_expand_tile(uint8_t *dst, const uint8_t *codes, const uint8_t *scales, int n_rows,
                                                int warp, int lane, const Kv4Lop &k) {
    constexpr int G = DH / KV4_GROUP, RPW = 32 / G, ROWS = 128 / W;     // rows of a warp at a time, and in all
    const int g = G == 4 ? (lane & 1) | ((lane >> 2) & 2) : lane & 1;
    const int r0 = G == 4 ? ((lane >> 1) & 3) | ((lane >> 4) << 2) : ((lane >> 1) & 3) | ((lane >> 3) << 2);
#pragma unroll
    for (int it = 0; it < ROWS / RPW; ++it) {
        const int r = warp * ROWS + it * RPW + r0;
        const uint4 w = *reinterpret_cast<const uint4 *>(codes + r * (DH / 2) + g * 16);
        uint32_t s = *reinterpret_cast<const uint16_t *>(scales + (r * G + g) * 2);
        if (r >= n_rows) s = 0;
        const uint32_t s2 = kv4_scale_pair(s), off2 = kv4_offset_pair(s2);
        uint8_t *row = dst + (g >> 1) * (128 * 128) + r * 128;
        const int c0 = (g & 1) * 4, x = r & 7;
        *reinterpret_cast<uint4 *>(row + (((c0 + 0) ^ x) << 4)) = kv4_expand(w.x, s2, off2, k);
        *reinterpret_cast<uint4 *>(row + (((c0 + 1) ^ x) << 4)) = kv4_expand(w.y, s2, off2, k);
        *reinterpret_cast<uint4 *>(row + (((c0 + 2) ^ x) << 4)) = kv4_expand(w.z, s2, off2, k);
        *reinterpret_cast<uint4 *>(row + (((c0 + 3) ^ x) << 4)) = kv4_expand(w.w, s2, off2, k);
    }
}

// One segment: steps [t0, t1) of a unit. Every role computes the same.
struct Kv4Seg {
    int b, h, q0, rows;          // item, head, first query row, rows of the unit that exist
    int t0, t1, len, n_valid;    // steps, the item's prefix rows, steps that hold keys
    int64_t next;                // first step behind the segment
    bool full;                   // the whole unit
};

__device__ __forceinline__ Kv4Seg kv4_segment(const Kv4TcArgs &p, int64_t at, int64_t end) {
    Kv4Seg s;
    const int unit = (int)(at / p.w.tiles);
    s.t0 = (int)(at - (int64_t)unit * p.w.tiles);
    s.t1 = (int)min((int64_t)p.w.tiles, s.t0 + (end - at));
    s.next = at + (s.t1 - s.t0);
    s.full = s.t0 == 0 && s.t1 == p.w.tiles;
    const int qt = unit % p.w.q_tiles, bh = unit / p.w.q_tiles;
    s.h = bh % p.a.c.H;
    s.b = bh / p.a.c.H;
    s.q0 = qt * p.w.unit_rows;
    s.rows = min(p.w.unit_rows, p.a.n_q - s.q0);
    s.len = kv4_len(p.a.c, p.a.prefix_len, p.a.shared ? 0 : s.b);
    const int tp = min(p.w.tiles_p, (s.len + 127) >> 7);              // prefix tiles that hold rows
    s.n_valid = max(0, min(s.t1, tp) - s.t0) + max(0, s.t1 - max(s.t0, p.w.tiles_p));
    return s;
}

// Steps of a segment that hold prefix rows; they come first.
__device__ __forceinline__ int kv4_prefix_steps(const Kv4TcArgs &p, const Kv4Seg &s) {
    return max(0, min(s.t1, min(p.w.tiles_p, (s.len + 127) >> 7)) - s.t0);
}

// Step number n (0 .. n_valid) of a segment: prefix tile (< tiles_p) or tail tile.
__device__ __forceinline__ int kv4_step_tile(const Kv4TcArgs &p, const Kv4Seg &s, int n) {
    const int in_prefix = kv4_prefix_steps(p, s);
    return n < in_prefix ? s.t0 + n : max(s.t0, p.w.tiles_p) + (n - in_prefix);
}

// Order of the 2 n loads of a segment: K0 K1 V0 K2 V1 .. V(n-1). A K tile is wanted
// one product earlier than the V tile of the step before it, which is only free when
// that step's weights are done. Returns 0 for K, 1 for V; j: the step in load order.
__device__ __forceinline__ int kv4_load_order(int i, int n, int &j) {
    const int v = i == 2 * n - 1 ? 1 : (i == 0 ? 0 : (i & 1) ^ 1);
    j = i == 2 * n - 1 ? n - 1 : (i == 0 ? 0 : (i & 1 ? (i + 1) >> 1 : (i >> 1) - 1));
    return v;
}
// Step that is loaded at position j: in the KH arrangement A0 B0 A1 B1 .. of the halves.
template <bool KH>
__device__ __forceinline__ int kv4_step_number(int j, int n) {
    return KH ? ((j & 1) ? ((n + 1) >> 1) + (j >> 1) : (j >> 1)) : j;
}

template <int DH, bool KH>    // KH: the halves share the rows and split the keys
__global__ void __launch_bounds__(512, 1)
    k_kv4_attn_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Kv4TcArgs p) {
    using namespace sm100;
    using C = Kv4AttnCfg<DH>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if (smem_u32(smem_raw) & 1023) {           // never expected; refuse rather than overrun
        if (threadIdx.x == 0) raise_device_error(p.a.err, DEV_ERR_LAYOUT);
        return;
    }
    uint8_t *smem = smem_raw;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *q_full = bars + 0, *q_empty = bars + 1;
    uint64_t *st_full = bars + 2, *st_empty = st_full + C::NS;      // staging ring
    uint64_t *k_full = st_empty + C::NS, *k_empty = k_full + 2;
    uint64_t *v_full = k_empty + 2, *v_empty = v_full + 2;
    uint64_t *s_full = v_empty + 2;            // [half]
    uint64_t *p_full = s_full + 2;             // [half][part]
    uint64_t *o_full = p_full + 4, *o_empty = o_full + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(o_empty + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert((2 + 2 * C::NS + 8 + 6 + 2) * 8 + 16 <= 256, "barrier region");
    float *stats = reinterpret_cast<float *>(smem + C::OFF_STATS);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(q_empty), 1);
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(smem_u32(&st_full[i]), 1);
            mbar_init(smem_u32(&st_empty[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&k_full[i]), 4);
            mbar_init(smem_u32(&k_empty[i]), 1);
            mbar_init(smem_u32(&v_full[i]), 4);
            mbar_init(smem_u32(&v_empty[i]), 1);
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&p_full[2 * i]), 128);
            mbar_init(smem_u32(&p_full[2 * i + 1]), 128);
        }
        mbar_init(smem_u32(o_full), 1);
        mbar_init(smem_u32(o_empty), 256);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 12) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t tmem_base = *tmem_slot;
    const int64_t w_lo = kv4_work_begin(p.w, blockIdx.x), w_hi = kv4_work_begin(p.w, blockIdx.x + 1);

    if (warp >= 12) {
        reg_dec<56>();
        if (warp == 12) {
            // ------------------------------------------------------------ UMMA issuer
            // per segment: S_A0 S_B0 | PV_A0 S_A1 PV_B0 S_B1 | PV_A1 S_A2 PV_B1 S_B2 | ...
            constexpr uint32_t idesc_s = idesc_bf16_f32(C::BQ, C::BK);
            constexpr uint32_t idesc_o = idesc_bf16_f32(C::BQ, DH, true);
            constexpr uint32_t BOX_UNITS = (C::BK * 128) >> 4, KV_UNITS = C::KV_BYTES >> 4;
            const uint64_t dq0 = sdesc_kmajor_sw128(smem_u32(smem + C::OFF_Q));
            const uint64_t dk0 = sdesc_kmajor_sw128(smem_u32(smem + C::OFF_K));
            const uint64_t dv0 = sdesc_mnmajor_sw128(smem_u32(smem + C::OFF_V), C::BK * 128);
            const bool leader = elect_one();
            auto wait_warp = [&](uint64_t *bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag, p.a.err) ? 1 : 0) != 0;
            };
            uint32_t nk = 0, nv = 0, np[2] = {0, 0}, sg = 0;     // ring positions, P tiles used, segments
            // last: no other half reads this K stage
            auto issue_s = [&](int h, bool last) -> bool {
                const uint32_t s = nk & 1;
                if (!wait_warp(&k_full[s], (nk >> 1) & 1)) return false;
                tc_fence_after();
                if (leader) {
                    const uint64_t dk = dk0 + s * KV_UNITS, dq = dq0 + (KH ? 0 : h) * (C::Q_BYTES >> 4);
#pragma unroll
                    for (int k = 0; k < DH / 16; ++k) {
                        const uint32_t off = (k >> 2) * BOX_UNITS + (k & 3) * 2;
                        umma_f16(tmem_base + h * 128, dq + off, dk + off, idesc_s, k > 0 ? 1u : 0u);
                    }
                    umma_commit(smem_u32(&s_full[h]));
                    if (last) umma_commit(smem_u32(&k_empty[s]));
                }
                __syncwarp();
                if (last) ++nk;
                return true;
            };
            auto issue_pv = [&](int h, bool first, bool last) -> bool {
                const uint32_t ph = np[h] & 1;
                if (!wait_warp(&p_full[2 * h], ph)) return false;
                const uint32_t s = nv & 1;
                if (!wait_warp(&v_full[s], (nv >> 1) & 1)) return false;
                tc_fence_after();
                const uint64_t dv = dv0 + s * KV_UNITS;
                constexpr int KSTEPS = C::BK / 16;
                if (leader) {
#pragma unroll
                    for (int k = 0; k < KSTEPS / 2; ++k)
                        umma_f16_ts(tmem_base + 256 + h * DH, tmem_base + h * 128 + k * 8, dv + k * 128, idesc_o,
                                    (!first || k > 0) ? 1u : 0u);
                }
                __syncwarp();
                if (!wait_warp(&p_full[2 * h + 1], ph)) return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = KSTEPS / 2; k < KSTEPS; ++k)
                        umma_f16_ts(tmem_base + 256 + h * DH, tmem_base + h * 128 + k * 8, dv + k * 128, idesc_o,
                                    1u);
                    if (last) umma_commit(smem_u32(&v_empty[s]));
                }
                __syncwarp();
                ++np[h];
                if (last) ++nv;
                return true;
            };
            bool ok = true;
            for (int64_t at = w_lo; at < w_hi && ok; ++sg) {
                const Kv4Seg seg = kv4_segment(p, at, w_hi);
                at = seg.next;
                const int nA = KH ? (seg.n_valid + 1) >> 1 : seg.n_valid;
                const int nB = KH ? seg.n_valid >> 1 : (seg.rows > 128 ? seg.n_valid : 0);
                ok = wait_warp(q_full, sg & 1);
                if (nA > 0) {
                    ok = ok && issue_s(0, KH || nB == 0);
                    if (nB > 0) ok = ok && issue_s(1, true);
                    // the epilogue of the segment before has read its O
                    if (sg > 0) ok = ok && wait_warp(o_empty, (sg - 1) & 1);
                    tc_fence_after();
                    for (int j = 0; j < nA && ok; ++j) {
                        ok = issue_pv(0, j == 0, KH || nB == 0);
                        if (ok && j + 1 < nA) ok = issue_s(0, KH || nB == 0);
                        if (ok && j < nB) {
                            ok = issue_pv(1, j == 0, true);
                            if (ok && j + 1 < nB) ok = issue_s(1, true);
                        }
                    }
                } else if (sg > 0) {
                    ok = ok && wait_warp(o_empty, (sg - 1) & 1);
                }
                if (ok && leader) {
                    umma_commit(smem_u32(q_empty));
                    umma_commit(smem_u32(o_full));
                }
                __syncwarp();
            }
        } else if (warp == 13 && lane == 0) {
            // ------------------------------------------------------------ codes and scales
            uint32_t n = 0;
            bool ok = true;
            for (int64_t at = w_lo; at < w_hi && ok;) {
                const Kv4Seg seg = kv4_segment(p, at, w_hi);
                at = seg.next;
                for (int i = 0; i < 2 * seg.n_valid && ok; ++i) {
                    int j;
                    const int which = kv4_load_order(i, seg.n_valid, j);
                    const int tile = kv4_step_tile(p, seg, kv4_step_number<KH>(j, seg.n_valid));
                    if (tile >= p.w.tiles_p) continue;
                    const uint32_t s = n % C::NS;
                    ok = mbar_wait(smem_u32(&st_empty[s]), ((n / C::NS) & 1) ^ 1, abort_flag, p.a.err);
                    if (!ok) break;
                    const int64_t row = kv4_row0(p.a.c, p.a.layer, which, p.a.shared ? 0 : seg.b, seg.h) +
                                        (int64_t)tile * 128;
                    const uint32_t bar = smem_u32(&st_full[s]);
                    const uint32_t dst = smem_u32(smem + C::OFF_ST + s * C::STAGE_BYTES);
                    mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
                    bulk_load(dst, p.a.base + row * (DH / 2), C::CODE_BYTES, bar);
                    bulk_load(dst + C::CODE_BYTES, p.a.base + p.a.c.scales_off + row * (C::G * 2), C::SCALE_BYTES, bar);
                    ++n;
                }
            }
        } else if (warp == 14 && lane == 0) {
            // ------------------------------------------------------------ Q
            uint32_t sg = 0;
            for (int64_t at = w_lo; at < w_hi; ++sg) {
                const Kv4Seg seg = kv4_segment(p, at, w_hi);
                at = seg.next;
                if (sg > 0 && !mbar_wait(smem_u32(q_empty), (sg - 1) & 1, abort_flag, p.a.err)) break;
                const int halves = !KH && seg.rows > 128 ? 2 : 1;
                const uint32_t qb = smem_u32(q_full);
                mbar_arrive_expect_tx(qb, halves * C::Q_BYTES);
                for (int h = 0; h < halves; ++h)
                    for (int x = 0; x < C::BOXES; ++x)
                        tma_load_4d(smem_u32(smem + C::OFF_Q + h * C::Q_BYTES + x * (C::BQ * 128)), &tmQ, qb,
                                    seg.h * DH + x * 64, seg.q0 + h * 128, seg.b, 0);
            }
        }
    } else if (warp >= 8) {
        // ---------------------------------------------------------------- K/V producers
        reg_dec<72>();
        uint32_t n = 0, st = 0;                     // tiles of each ring, staged tiles
        bool ok = true;
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag, p.a.err) ? 1 : 0) != 0;
        };
        for (int64_t at = w_lo; at < w_hi && ok;) {
            const Kv4Seg seg = kv4_segment(p, at, w_hi);
            at = seg.next;
#pragma unroll 1
            for (int i = 0; i < 2 * seg.n_valid; ++i) {
                int j;
                const int which = kv4_load_order(i, seg.n_valid, j);
                const int tile = kv4_step_tile(p, seg, kv4_step_number<KH>(j, seg.n_valid));
                const uint32_t s = (n + j) & 1, par = (((n + j) >> 1) & 1) ^ 1;
                uint64_t *full = which ? &v_full[s] : &k_full[s], *empty = which ? &v_empty[s] : &k_empty[s];
                uint8_t *dst = smem + (which ? C::OFF_V : C::OFF_K) + s * C::KV_BYTES;
                if (!(ok = wait_all(empty, par))) break;
                if (tile < p.w.tiles_p) {
                    const uint32_t ss = st % C::NS;
                    if (!(ok = wait_all(&st_full[ss], (st / C::NS) & 1))) break;
                    const uint8_t *stage = smem + C::OFF_ST + ss * C::STAGE_BYTES;
                    kv4_expand_tile<DH, 4>(dst, stage, stage + C::CODE_BYTES, seg.len - tile * 128, warp - 8, lane,
                                           p.a.lop);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&st_empty[ss]));
                        mbar_arrive(smem_u32(full));
                    }
                    ++st;
                } else if (lane == 0) {
                    const uint32_t bar = smem_u32(full);
                    if (warp == 8) {
                        mbar_arrive_expect_tx(bar, C::KV_BYTES);
                        for (int x = 0; x < C::BOXES; ++x)
                            tma_load_4d(smem_u32(dst + x * (C::BK * 128)), which ? &tmV : &tmK, bar, seg.h * DH + x * 64,
                                        (tile - p.w.tiles_p) * 128, seg.b, 0);
                    } else {
                        mbar_arrive(bar);
                    }
                }
            }
            n += seg.n_valid;
        }
    } else {
        // ---------------------------------------------------------------- softmax (warps 0..7)
        reg_inc<192>();
        const int h = warp >> 2, quad = warp & 3, r = quad * 32 + lane;    // TMEM lane = row of the half
        const uint32_t t_lane = tmem_base + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_s = t_lane + h * 128, t_o = t_lane + 256 + h * DH;
        const float c = p.a.scale_log2;
        bool ok = true;
        uint32_t ns = 0, sg = 0;
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag, p.a.err) ? 1 : 0) != 0;
        };
        for (int64_t at = w_lo; at < w_hi; ++sg) {
            const bool first_seg = at == w_lo;
            const Kv4Seg seg = kv4_segment(p, at, w_hi);
            at = seg.next;
            const int nA = KH ? (seg.n_valid + 1) >> 1 : seg.n_valid;
            const int nB = KH ? seg.n_valid >> 1 : (seg.rows > 128 ? seg.n_valid : 0);
            const int nt = h ? nB : nA, n0 = KH && h ? nA : 0;
            // keys of step n: (n < n_pre ? keys_p : keys_t) - 128 n
            const int n_pre = kv4_prefix_steps(p, seg), keys_p = seg.len - (seg.t0 + n0) * C::BK;
            const int keys_t = p.a.n_tail - (max(seg.t0, p.w.tiles_p) - p.w.tiles_p - n_pre + n0) * C::BK;
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = 0; j < nt && ok; ++j, ++ns) {
                if (!(ok = wait_all(&s_full[h], ns & 1))) break;
                tc_fence_after();
                float sv[4][32];                          // S row: key 32a+b in sv[a][b]
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) tmem_ld32(t_s + cc * 32, sv[cc]);
                tmem_wait_ld();
                const int n_keys = (n0 + j < n_pre ? keys_p : keys_t) - j * C::BK;
                if (n_keys < C::BK) {
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (i >= n_keys) sv[i >> 5][i & 31] = -INFINITY;
                }
                float m4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m4[i] = fmaxf(sv[0][2 * i], sv[0][2 * i + 1]);
#pragma unroll
                for (int i = 8; i < 128; i += 2)
                    m4[(i >> 1) & 3] = fmax3(m4[(i >> 1) & 3], sv[i >> 5][i & 31], sv[i >> 5][(i + 1) & 31]);
                const float mx = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
                // move the running max only when this tile raises it by more than 2^8
                const bool first = (m_run == -INFINITY);
                const bool grow = first || (mx - m_run) * c > kRescaleLog2;
                const float m_new = grow ? fmaxf(m_run, mx) : m_run;
                const float alpha = (grow && !first) ? ex2_approx((m_run - m_new) * c) : 1.f;
                l_run *= alpha;
                m_run = m_new;
                const float mc = m_run == -INFINITY ? 0.f : m_run * c;
                uint64_t s4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) s4[i] = 0ull;
                const uint64_t c2 = f2_pack(c, c), nmc2 = f2_pack(-mc, -mc);
                auto signal_p = [&](int part) {
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(smem_u32(&p_full[2 * h + part]));
                };
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t u[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        float x0, x1, e0, e1;
                        f2_unpack(f2_fma(f2_pack(sv[cc][2 * q], sv[cc][2 * q + 1]), c2, nmc2), x0, x1);
                        // all on the MUFU units: with every 8th pair on the FMA pipe the
                        // expansion has less of the issue slots (175 us against 157; 256 rows,
                        // 32 heads of 128, P 33792). A NaN score makes its row's sum one.
                        e0 = ex2_approx(x0);
                        e1 = ex2_approx(x1);
                        s4[q & 3] = f2_add(s4[q & 3], f2_pack(e0, e1));
                        u[q] = pack_bf16x2(e0, e1);
                    }
                    tmem_st16(t_s + cc * 16, u);               // P_h: keys 32cc .. 32cc+31
                    if (cc == 1) {
                        // O rescale (rare) before the first P signal; O_h holds PV_h of the
                        // tiles before this one (complete: S_h was issued after them)
                        if (__any_sync(0xffffffffu, grow && !first)) {
                            float ov[32];
#pragma unroll
                            for (int oc = 0; oc < DH / 32; ++oc) {
                                tmem_ld32(t_o + oc * 32, ov);
                                tmem_wait_ld();
                                uint32_t w32[32];
#pragma unroll
                                for (int i = 0; i < 32; ++i) w32[i] = __float_as_uint(ov[i] * alpha);
                                tmem_st32(t_o + oc * 32, w32);
                            }
                        }
                        signal_p(0);
                    }
                }
                signal_p(1);
                const uint64_t s2 = f2_add(f2_add(s4[0], s4[1]), f2_add(s4[2], s4[3]));
                float sa, sb;
                f2_unpack(s2, sa, sb);
                l_run += sa + sb;
            }
            // -------------------------------------------------------- epilogue of the segment
            // KH: the halves' results are merged, half h writing the columns of its half;
            // else half h writes its own rows.
            float m = m_run, fA = 0.f, fB = 0.f, l = l_run;
            if (KH) {
                float *st = stats + (sg & 1) * (4 * C::BQ);
                st[(2 * h + 0) * C::BQ + r] = m_run;
                st[(2 * h + 1) * C::BQ + r] = l_run;
                softmax_bar_sync();
                const float mA = st[r], lA = st[C::BQ + r], mB = st[2 * C::BQ + r], lB = st[3 * C::BQ + r];
                m = fmaxf(mA, mB);
                const float mz = m == -INFINITY ? 0.f : m;
                const float wA = ex2_approx((mA - mz) * c), wB = nB > 0 ? ex2_approx((mB - mz) * c) : 0.f;
                l = lA * wA + (nB > 0 ? lB * wB : 0.f);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                fA = wA * inv;
                fB = wB * inv;
            } else {
                fA = l == 0.f ? 0.f : 1.f / l;
            }
            const int row = seg.q0 + (KH ? 0 : h * 128) + r;       // query row of this thread
            const bool live = (KH ? r : h * 128 + r) < seg.rows;
            const float lse2 = l == 0.f ? -INFINITY : m * c + log2f(l);
            const int slot = 2 * (int)blockIdx.x + (first_seg ? 0 : 1);
            const int64_t prow = (int64_t)slot * p.w.slot_rows + (KH ? 0 : h * 128) + r;
            if (live && (!KH || h == 0)) {
                if (!seg.full)
                    p.part_l[prow] = lse2;
                else if (p.a.lse)
                    p.a.lse[((int64_t)seg.h * p.a.B + seg.b) * p.a.n_q + row] = lse2 * KV4_LN2;
            }
            ok = ok && wait_all(o_full, sg & 1);
            if (ok && (KH || h == 0 || seg.rows > 128)) {
                tc_fence_after();
                constexpr int COLS = KH ? DH / 2 : DH;
                const int col0 = KH ? h * COLS : 0;
                bf16 *dst = (bf16 *)p.a.out + ((int64_t)seg.b * p.a.n_q + row) * ((int64_t)p.a.c.H * DH) + seg.h * DH;
                float *pdst = p.part_o + prow * DH;
#pragma unroll
                for (int cc = 0; cc < COLS / 32; ++cc) {
                    const int col = col0 + cc * 32;
                    float oa[32];
                    if (seg.n_valid > 0) {                     // else nothing was written to O
                        tmem_ld32(KH ? t_lane + 256 + col : t_o + col, oa);
                        if (KH && nB > 0) {
                            float ob[32];
                            tmem_ld32(t_lane + 256 + DH + col, ob);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) oa[i] = fmaf(fA, oa[i], fB * ob[i]);
                        } else {
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) oa[i] *= fA;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) oa[i] = 0.f;
                    }
                    if (live && seg.full) store_bf16x32(dst + col, oa);
                    if (live && !seg.full) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<float4 *>(pdst + col)[i] =
                                make_float4(oa[4 * i], oa[4 * i + 1], oa[4 * i + 2], oa[4 * i + 3]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(o_empty));
            // after a failed wait the remaining segments are walked without any wait, so
            // that both halves pass the same number of softmax_bar_sync()
        }
    }
    tc_fence_before();
    __syncthreads();
    settle_if_aborted(abort_flag);
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// Join the partial results of the units that the sharing cut. Block y stands for
// the boundary in front of CTA y + 1: where it is the first one inside a unit, its
// warps go through the CTAs that share the unit, in order, four query rows at a time.
constexpr int KV4_JOIN_ROWS = 4;

template <int DH>
__global__ void __launch_bounds__(256) k_kv4_join(const __grid_constant__ Kv4TcArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int R = KV4_JOIN_ROWS, C = DH / 32;
    const int c1 = blockIdx.y + 1, T = p.w.tiles;
    const int64_t edge = kv4_work_begin(p.w, c1);
    const int unit = (int)(edge / T);
    const int64_t begin = (int64_t)unit * T, end = begin + T;
    if (edge == begin || kv4_work_begin(p.w, c1 - 1) > begin) return;   // not inside, or not the first
    const int lane = threadIdx.x & 31, r0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * R;
    const int qt = unit % p.w.q_tiles, bh = unit / p.w.q_tiles, h = bh % p.a.c.H, b = bh / p.a.c.H;
    const int row0 = qt * p.w.unit_rows + r0, live = min(min(R, p.w.unit_rows - r0), p.a.n_q - row0);
    if (live <= 0) return;
    float m[R], sum[R], o[R][C];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        m[k] = -INFINITY;
        sum[k] = 0.f;
#pragma unroll
        for (int j = 0; j < C; ++j) o[k][j] = 0.f;
    }
    // The CTAs that share the unit, one a lane (32 at a time): CTA c's partial result is
    // in its slot 0 (its first segment) unless the unit begins inside its range.
    for (int c0 = c1 - 1; c0 < p.w.grid && kv4_work_begin(p.w, c0) < end; c0 += 32) {
        const int c = c0 + lane;
        const int64_t lo = kv4_work_begin(p.w, c);
        const bool in = c < p.w.grid && lo < end;
        const int slot = 2 * c + (lo < begin ? 1 : 0);
        const int n = __popc(__ballot_sync(0xffffffffu, in));
        float w[R];
#pragma unroll
        for (int k = 0; k < R; ++k)
            w[k] = in && k < live ? p.part_l[(int64_t)slot * p.w.slot_rows + r0 + k] : -INFINITY;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const float mn = fmaxf(m[k], warp_max(w[k])), mz = mn == -INFINITY ? 0.f : mn;
            const float scale = exp2f(m[k] - mz);              // of what earlier ones gave
            w[k] = in ? exp2f(w[k] - mz) : 0.f;
            m[k] = mn;
            sum[k] = sum[k] * scale + warp_sum(w[k]);
#pragma unroll
            for (int j = 0; j < C; ++j) o[k][j] *= scale;
        }
        for (int i = 0; i < n; ++i) {
            const float *src = p.part_o + ((int64_t)__shfl_sync(0xffffffffu, slot, i) * p.w.slot_rows + r0) * DH + lane;
            float v[R][C];
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int j = 0; j < C; ++j) v[k][j] = k < live ? src[k * DH + 32 * j] : 0.f;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const float wi = __shfl_sync(0xffffffffu, w[k], i);
#pragma unroll
                for (int j = 0; j < C; ++j) o[k][j] = fmaf(wi, v[k][j], o[k][j]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        if (k >= live) continue;
        const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
        bf16 *dst = (bf16 *)p.a.out + ((int64_t)b * p.a.n_q + row0 + k) * ((int64_t)p.a.c.H * DH) + h * DH;
#pragma unroll
        for (int j = 0; j < C; ++j) dst[lane + 32 * j] = __float2bfloat16_rn(o[k][j] * inv);
        if (p.a.lse && lane == 0)
            p.a.lse[((int64_t)h * p.a.B + b) * p.a.n_q + row0 + k] =
                sum[k] == 0.f ? -INFINITY : (m[k] + log2f(sum[k])) * KV4_LN2;
    }
}

}  // namespace qi21
