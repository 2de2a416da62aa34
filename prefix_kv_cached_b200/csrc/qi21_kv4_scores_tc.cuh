// Accumulated attention weight of the rows of a 4-bit prefix cache on tcgen05
// tensor cores (BF16 mode):
//   sum_j = sum_i 2^(c q_i . k_j - lse2_i),  c = log2(e) / sqrt(Dh).
//
// The products are formed transposed, S^T = K Q^T (M = 128 keys in the TMEM lanes,
// N = 128 queries in the columns): a thread then holds one key's row and the sum
// over queries stays in its registers, without a shuffle or an atomic. A CTA
// expands one 128-key tile of a head once and streams the query tiles past it
// (TMA, two stages); two S buffers let the next product run under the exponentials,
// and two CTAs share an SM so that one's loads of S and waits hide under the
// other's exponentials. Where the key tiles alone do not fill the SMs the queries
// are split over CTAs too, and k_kv4_scores_reduce adds their sums in order.
//   warps 0..7 : expand the K tile, then exponentials and sums: thread = key, warps
//                0..3 the first 64 queries of a tile, 4..7 the others (four such
//                warps an SMSP hide each other's TMEM loads and MUFU latency)
//   warp 8     : TMEM allocator + UMMA issuer
//   warp 9     : Q tiles by TMA and the queries' offsets -lse2
// Bound by the exponentials: 128 x 128 a tile take 1024 cycles of the SM's MUFU
// units, the product 512 tensor cycles (head_dim 128). KV4_SC_POLY of every 8 pairs
// therefore go to the FMA pipe. 164 us for 4096 queries, P 4608, 32 heads of 128 (940
// TFLOP/s); with the exponentials and sums left out it runs 104 us, the product's own
// time. One warpgroup of exponentials a CTA is as fast as the two here take with twice
// the rows in registers; loading S one key a thread (its 128 queries' offsets from
// shared memory) costs 27 us more.
#pragma once
#include "qi21_kv4_attn_tc.cuh"

namespace qi21 {

constexpr int KV4_SC_POLY = 2;   // us at the size above with 0 .. 3 of 8: 182, 170, 165, 173

template <int DH>
struct Kv4ScoreCfg {
    static constexpr int BK = 128, BQ = 128, BOXES = DH / 64, G = DH / KV4_GROUP;
    static constexpr int TILE_BYTES = 128 * DH * 2;
    static constexpr int OFF_K = 0, OFF_Q = TILE_BYTES, OFF_LSE = OFF_Q + 2 * TILE_BYTES;
    static constexpr int NL = 4;                              // stages of 128 offsets
    static constexpr int OFF_BAR = OFF_LSE + NL * 128 * 4;
    static constexpr int OFF_SUM = OFF_BAR + 256;            // [half][128] floats
    static constexpr size_t SMEM = (size_t)OFF_SUM + 2 * 128 * 4;
    static constexpr int THREADS = 320;
};

struct Kv4ScoreTcArgs {
    Kv4ScoreArgs a;
    int q_tiles, n_split;        // query tiles, parts they are split into
    float *part;                 // [n_split][B][H][Pp] when n_split > 1
};

// 2^x of a pair by a polynomial of degree 5 (exp2_poly_fit.py's fit of that degree,
// relative error 2e-7: these weights are a result in fp32), with 2^n as a factor: a NaN stays one, x > 128 gives +inf, x < -127 gives 0.
__device__ __forceinline__ uint64_t kv4_ex2_pair(uint64_t x2) {
    float x0, x1;
    f2_unpack(x2, x0, x1);
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x0) : "f"(x0), "f"(-127.f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x1) : "f"(x1), "f"(-127.f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x0) : "f"(x0), "f"(128.f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x1) : "f"(x1), "f"(128.f));
    auto two = [](float v) { return f2_pack(v, v); };
    const uint64_t magic = two(12582912.f);
    const uint64_t x = f2_pack(x0, x1), t = f2_add(x, magic), f = f2_sub(x, f2_sub(t, magic));
    uint64_t q = f2_fma(two(0.0013218672f), f, two(0.009671698f));
    q = f2_fma(q, f, two(0.05550893f));
    q = f2_fma(q, f, two(0.24022238f));
    q = f2_fma(q, f, two(0.6931469f));
    q = f2_fma(q, f, two(1.0f));
    float t0, t1;
    f2_unpack(t, t0, t1);
    const float n0 = __uint_as_float((__float_as_uint(t0) << 23) + 0x3F800000u);
    const float n1 = __uint_as_float((__float_as_uint(t1) << 23) + 0x3F800000u);
    uint64_t e;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(e) : "l"(q), "l"(f2_pack(n0, n1)));
    return e;
}

// grid (key tiles, H, B * n_split)
template <int DH>
__global__ void __launch_bounds__(320, 2)
    k_kv4_scores_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ Kv4ScoreTcArgs p) {
    using namespace sm100;
    using C = Kv4ScoreCfg<DH>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    if (smem_u32(smem_raw) & 1023) {           // never expected; refuse rather than overrun
        if (threadIdx.x == 0) raise_device_error(p.a.err, DEV_ERR_LAYOUT);
        return;
    }
    uint8_t *smem = smem_raw;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *k_ready = bars, *q_full = bars + 1, *q_empty = q_full + 2, *s_full = q_empty + 2, *s_empty = s_full + 2;
    uint64_t *l_full = s_empty + 2, *l_empty = l_full + C::NL;       // offsets of the queries
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(l_empty + C::NL);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *lse_s = reinterpret_cast<float *>(smem + C::OFF_LSE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y, b = blockIdx.z / p.n_split, sp = blockIdx.z - b * p.n_split;
    const int k0 = blockIdx.x * C::BK;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(k_ready), 256);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&q_full[i]), 1);
            mbar_init(smem_u32(&q_empty[i]), 1);
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&s_empty[i]), 8);
        }
        for (int i = 0; i < C::NL; ++i) {
            mbar_init(smem_u32(&l_full[i]), 1);
            mbar_init(smem_u32(&l_empty[i]), 8);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t tmem_base = *tmem_slot;
    const int len = kv4_len(p.a.c, p.a.prefix_len, b);
    const int qt_lo = (int)((int64_t)sp * p.q_tiles / p.n_split), qt_hi = (int)((int64_t)(sp + 1) * p.q_tiles / p.n_split);
    const int nt = k0 < len ? qt_hi - qt_lo : 0;
    if (warp == 8) {
        // ---------------------------------------------------------------- UMMA issuer
        constexpr uint32_t idesc = idesc_bf16_f32(C::BK, C::BQ), BOX_UNITS = (128 * 128) >> 4;
        const uint64_t dk = sdesc_kmajor_sw128(smem_u32(smem + C::OFF_K));
        const uint64_t dq0 = sdesc_kmajor_sw128(smem_u32(smem + C::OFF_Q));
        const bool leader = elect_one();
        auto wait_warp = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag, p.a.err) ? 1 : 0) != 0;
        };
        bool ok = nt == 0 || wait_warp(k_ready, 0);
        for (int n = 0; n < nt && ok; ++n) {
            const int s = n & 1;
            const uint32_t ph = (n >> 1) & 1;
            ok = wait_warp(&q_full[s], ph) && wait_warp(&s_empty[s], ph ^ 1);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
                const uint64_t dq = dq0 + s * (C::TILE_BYTES >> 4);
#pragma unroll
                for (int k = 0; k < DH / 16; ++k) {
                    const uint32_t off = (k >> 2) * BOX_UNITS + (k & 3) * 2;
                    umma_f16(tmem_base + s * 128, dk + off, dq + off, idesc, k > 0 ? 1u : 0u);
                }
                umma_commit(smem_u32(&s_full[s]));
                umma_commit(smem_u32(&q_empty[s]));
            }
            __syncwarp();
        }
    } else if (warp == 9) {
        // ---------------------------------------------------------------- query tiles
        const float *lse = p.a.lse + ((int64_t)h * p.a.c.B + b) * p.a.n_q;
        float next[4];                              // the offsets one tile ahead
        auto fetch = [&](int q0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = q0 + i * 32 + lane;
                next[i] = row < p.a.n_q ? lse[row] : -INFINITY;
            }
        };
        if (nt > 0) fetch(qt_lo * C::BQ);
        for (int n = 0; n < nt; ++n) {
            // a Q stage is free once its product is done, under the exponentials; the
            // offsets have a ring of their own
            const int s = n & 1, sl = n % C::NL, q0 = (qt_lo + n) * C::BQ;
            bool ok = mbar_wait(smem_u32(&q_empty[s]), ((n >> 1) & 1) ^ 1, abort_flag, p.a.err);
            if (!__all_sync(0xffffffffu, ok ? 1 : 0)) break;
            if (lane == 0) {
                const uint32_t qb = smem_u32(&q_full[s]);
                mbar_arrive_expect_tx(qb, C::TILE_BYTES);
                for (int x = 0; x < C::BOXES; ++x)
                    tma_load_4d(smem_u32(smem + C::OFF_Q + s * C::TILE_BYTES + x * (C::BQ * 128)), &tmQ, qb,
                                h * DH + x * 64, q0, b, 0);
            }
            ok = mbar_wait(smem_u32(&l_empty[sl]), ((n / C::NL) & 1) ^ 1, abort_flag, p.a.err);
            if (!__all_sync(0xffffffffu, ok ? 1 : 0)) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) lse_s[sl * 128 + i * 32 + lane] = -kv4_lse2(next[i]);
            fetch(q0 + C::BQ);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&l_full[sl]));
        }
    } else {
        // ---------------------------------------------------------------- expand, then sum
        const int half = warp >> 2, quad = warp & 3;
        float *sums = reinterpret_cast<float *>(smem + C::OFF_SUM) + half * 128;   // [half][key of the tile]
        if (nt > 0) {
            const int64_t row = kv4_row0(p.a.c, p.a.layer, 0, b, h) + k0;
            kv4_expand_tile<DH, 8>(smem + C::OFF_K, p.a.base + row * (DH / 2),
                                   p.a.base + p.a.c.scales_off + row * (C::G * 2), len - k0, warp, lane, p.a.lop);
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(k_ready));
            const uint32_t t_s = tmem_base + ((uint32_t)(quad * 32) << 16) + half * 64;
            const uint64_t c2 = f2_pack(p.a.scale_log2, p.a.scale_log2);
            auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag, p.a.err) ? 1 : 0) != 0;
            };
            // a thread's four keys of the quadrant's 32: lane / 4 + 8 k; of every 8 queries
            // two, at 2 (lane % 4), so that one load of their offsets serves four keys
            uint64_t total[4] = {0ull, 0ull, 0ull, 0ull};       // pairs of +0.f
            for (int n = 0; n < nt; ++n) {
                const int s = n & 1, sl = n % C::NL;
                if (!wait_all(&s_full[s], (n >> 1) & 1) || !wait_all(&l_full[sl], (n / C::NL) & 1)) break;
                tc_fence_after();
                float sv[2][32];
                tmem_ld16x256_64(t_s + s * 128, sv[0]);
                tmem_ld16x256_64(t_s + s * 128 + (16u << 16), sv[1]);
                uint64_t off[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    off[i] = *reinterpret_cast<const uint64_t *>(lse_s + sl * 128 + half * 64 + i * 8 + 2 * (lane & 3));
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&s_empty[s]));
                    mbar_arrive(smem_u32(&l_empty[sl]));
                }
                uint64_t part[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = 4 * i + 2 * (k & 1);
                        const uint64_t x = f2_fma(f2_pack(sv[k >> 1][at], sv[k >> 1][at + 1]), c2, off[i]);
                        uint64_t e;
                        if ((i * 4 + k) % 8 >= 8 - KV4_SC_POLY) {
                            e = kv4_ex2_pair(x);
                        } else {
                            float x0, x1;
                            f2_unpack(x, x0, x1);
                            e = f2_pack(ex2_approx(x0), ex2_approx(x1));
                        }
                        part[k] = f2_add(part[k], e);
                    }
#pragma unroll
                for (int k = 0; k < 4; ++k) total[k] = f2_add(total[k], part[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float a, c;
                f2_unpack(total[k], a, c);
                a += c;
                a += __shfl_xor_sync(0xffffffffu, a, 1);
                a += __shfl_xor_sync(0xffffffffu, a, 2);
                if ((lane & 3) == 0) sums[quad * 32 + k * 8 + (lane >> 2)] = a;
            }
        } else {
            sums[quad * 32 + lane] = 0.f;
        }
        softmax_bar_sync();                                     // warps 0..7
        const int j = k0 + (int)threadIdx.x;
        if (half == 0) {
            const int64_t at = ((int64_t)b * p.a.c.H + h) * p.a.c.P + j;
            const float sum = sums[threadIdx.x] + sums[128 + threadIdx.x];   // the halves, in one order
            if (p.n_split > 1) {
                if (j < len) p.part[(((int64_t)sp * p.a.c.B + b) * p.a.c.H + h) * p.a.c.Pp + j] = sum;
            } else if (j < p.a.c.P && (j < len || p.a.out != p.a.in)) {
                p.a.out[at] = (p.a.in ? p.a.in[at] : 0.f) + (j < len ? sum : 0.f);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    settle_if_aborted(abort_flag);
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 256);
    }
}

// out = in + the parts' sums, in order; entries behind an item's rows are copied.
static __global__ void __launch_bounds__(256) k_kv4_scores_reduce(Kv4ScoreTcArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int j = blockIdx.x * 256 + threadIdx.x, h = blockIdx.y, b = blockIdx.z;
    if (j >= p.a.c.P) return;
    const int64_t at = ((int64_t)b * p.a.c.H + h) * p.a.c.P + j;
    const bool live = j < kv4_len(p.a.c, p.a.prefix_len, b);
    if (!live && p.a.out == p.a.in) return;
    float sum = 0.f;
    if (live)
        for (int s = 0; s < p.n_split; ++s) sum += p.part[(((int64_t)s * p.a.c.B + b) * p.a.c.H + h) * p.a.c.Pp + j];
    p.a.out[at] = (p.a.in ? p.a.in[at] : 0.f) + sum;
}

}  // namespace qi21
