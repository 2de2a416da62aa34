// Attention and accumulated weights over a 4-bit prefix cache for a few query rows
// (BF16 mode): the calls whose time is that of reading the cache once.
//
// A warp streams 64-key chunks of one head through a ring of its own (bulk copies,
// no other warp to wait for) and never writes an expanded value to
// memory: the codes become the register operands of mma.sync m16n8k16 with the
// cache as the 16-row operand and 8 queries as the columns,
//   S^T (16 keys x 8 queries)  = K Q^T   over the dims,
//   O^T (16 dims x 8 queries) += V^T P^T over the keys.
// Both operands' index orders are free as long as the two sides agree, and are
// chosen so that a code word needs no rearrangement:
//   * thread t of a quad holds dims [t Dh/4, (t+1) Dh/4) of its keys: whole code
//     words, a single scale; the pairs of the products' k index are nibbles i and
//     i + 4 of a word (Q is permuted alike, once);
//   * thread group g holds dims [g Dh/8, (g+1) Dh/8) of V; the halves of the words
//     of keys 2t and 2t + 1 side by side give pairs along the keys, with a pair of
//     scales; nibble i of them is row g of product tile i.
// P^T comes from S^T by packing to bf16 and a transposing 8 x 8 move. Softmax per
// chunk, in fp32, the running maximum per query; the warps of a CTA are merged
// through shared memory and up to KV4R_CLUSTER key splits through the shared memory of a
// cluster (else by k_kv4_combine), in a fixed order.
// (tcgen05 would want the expanded cache in shared memory: 2 bytes an element
// written and read again, which alone is as long as the read of 4.5 bits from HBM.)
// The weights are rounded to bf16 for the product with V (2^-8 of each at most): its
// operands have one type, and V's values are exact in bf16. Sums, maxima and outputs are
// fp32.
// Bound by latency: a scheduler has three warps, and each is a single chain of expansion,
// product, maximum over shuffles, exponentials, transpose, expansion and product. 16 keys
// of K and V at head_dim 128 take 575 cycles, of which the 159 instructions of the
// expansion on the ALU pipe at half rate fill 318 (ALU 49 %, issue slots 52 %): 50 us for
// one row over P 33792, 32 heads of 128 (3.1 TB/s), of which the pass over the key
// splits' results takes some 8; the loads alone run 29 us, HBM's own time is 24.
#pragma once
#include "qi21_kv4_attn_tc.cuh"

namespace qi21 {

constexpr int KV4R_CHUNK = 64, KV4R_WARPS = 4, KV4R_M = KV4R_CHUNK / 16;   // product tiles of keys a chunk
constexpr int KV4R_CLUSTER = KV4_ROWS_CLUSTER;

template <int DH, bool V>      // V: with the value rows
struct Kv4RowsCfg {
    static constexpr int G = DH / KV4_GROUP;
    static constexpr int CODES = KV4R_CHUNK * DH / 2, SCALES = KV4R_CHUNK * G * 2;
    static constexpr int STAGE = (V ? 2 : 1) * (CODES + SCALES);
    static constexpr int STAGES = V ? 2 : 3;
    static constexpr int OFF_BAR = KV4R_WARPS * STAGES * STAGE;
    static constexpr size_t SMEM = (size_t)OFF_BAR + KV4R_WARPS * STAGES * 8 + 16;
};

// ORDERED: kept in program order, which keeps the operands of later products out of
// the registers.
template <bool ORDERED = false>
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if (ORDERED)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// The pairs (dims i, i + 4) of 8 bf16 values, the order in which a code word unfolds.
__device__ __forceinline__ void kv4_order(uint4 u, uint32_t (&p)[4]) {
    p[0] = __byte_perm(u.x, u.z, 0x5410);
    p[1] = __byte_perm(u.x, u.z, 0x7632);
    p[2] = __byte_perm(u.y, u.w, 0x5410);
    p[3] = __byte_perm(u.y, u.w, 0x7632);
}

// One warp's ring over the chunks of its share.
template <int DH, bool V>
struct Kv4Ring {
    using C = Kv4RowsCfg<DH, V>;
    uint8_t *stages;
    uint64_t *bars;
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;   // of the head
    __device__ __forceinline__ void load(int n, int chunk) const {           // one lane
        const int s = n % C::STAGES;
        const uint32_t dst = sm100::smem_u32(stages + s * C::STAGE), bar = sm100::smem_u32(&bars[s]);
        const int64_t r = (int64_t)chunk * KV4R_CHUNK;
        sm100::mbar_arrive_expect_tx(bar, C::STAGE);
        bulk_load(dst, k_codes + r * (DH / 2), C::CODES, bar);
        bulk_load(dst + C::CODES, k_scales + r * (C::G * 2), C::SCALES, bar);
        if (V) {
            bulk_load(dst + C::CODES + C::SCALES, v_codes + r * (DH / 2), C::CODES, bar);
            bulk_load(dst + 2 * C::CODES + C::SCALES, v_scales + r * (C::G * 2), C::SCALES, bar);
        }
    }
};

// Q operands of NT tiles of 8 queries from row q0 on: bq[tile][step][2]; rows behind
// n_q are zeros.
template <int DH, int NT>
__device__ __forceinline__ void kv4_load_q(const bf16 *q, int q0, int n_q, int64_t d, int g, int t,
                                           uint32_t (&bq)[NT][DH / 16][2]) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int row = q0 + 8 * j + g;
#pragma unroll
        for (int w = 0; w < DH / 32; ++w) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (row < n_q) u = *reinterpret_cast<const uint4 *>(q + row * d + t * (DH / 4) + w * 8);
            uint32_t p[4];
            kv4_order(u, p);
            bq[j][2 * w][0] = p[0];
            bq[j][2 * w][1] = p[1];
            bq[j][2 * w + 1][0] = p[2];
            bq[j][2 * w + 1][1] = p[3];
        }
    }
}

// S^T of 16 keys from their K operands: ka, kb the pairs of keys g and g + 8, word by word.
template <int DH, int NT>
__device__ __forceinline__ void kv4_scores_step(const uint32_t (&ka)[4], const uint32_t (&kb)[4], int w,
                                                const uint32_t (&bq)[NT][DH / 16][2], float (&s)[NT][4]) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        mma_bf16(s[j], ka[0], kb[0], ka[1], kb[1], bq[j][2 * w][0], bq[j][2 * w][1]);
        mma_bf16(s[j], ka[2], kb[2], ka[3], kb[3], bq[j][2 * w + 1][0], bq[j][2 * w + 1][1]);
    }
}

// S^T of MM tiles of 16 keys from row r of a staged chunk. The tiles take turns, so
// that a product does not wait for the one before it.
template <int DH, int NT, int MM, bool ORDERED = false>
__device__ __forceinline__ void kv4_scores_staged(const uint8_t *codes, const uint8_t *scales, int r, int g, int t,
                                                  const uint32_t (&bq)[NT][DH / 16][2], const Kv4Lop &k,
                                                  float (*s)[NT][4]) {
    constexpr int G = DH / KV4_GROUP, W = DH / 32;
    alignas(16) uint32_t wd[MM][2][W];             // code words of keys g and g + 8
    uint32_t sc[MM][2], of[MM][2];
    const int grp = t * G / 4;
#pragma unroll
    for (int m = 0; m < MM; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = r + 16 * m + 8 * i + g;
            const uint8_t *src = codes + row * (DH / 2) + t * (DH / 8);
            if (DH == 128) *reinterpret_cast<uint4 *>(wd[m][i]) = *reinterpret_cast<const uint4 *>(src);
            else *reinterpret_cast<uint2 *>(wd[m][i]) = *reinterpret_cast<const uint2 *>(src);
            sc[m][i] = kv4_scale_pair(*reinterpret_cast<const uint16_t *>(scales + (row * G + grp) * 2));
            of[m][i] = kv4_offset_pair(sc[m][i]);
        }
#pragma unroll
    for (int m = 0; m < MM; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[m][j][i] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        uint32_t ka[MM][4], kb[MM][4];
#pragma unroll
        for (int m = 0; m < MM; ++m) {
            kv4_pairs(wd[m][0][w], sc[m][0], of[m][0], k, ka[m]);
            kv4_pairs(wd[m][1][w], sc[m][1], of[m][1], k, kb[m]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int m = 0; m < MM; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    mma_bf16<ORDERED>(s[m][j], ka[m][2 * i], kb[m][2 * i], ka[m][2 * i + 1], kb[m][2 * i + 1],
                             bq[j][2 * w + i][0], bq[j][2 * w + i][1]);
    }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// Four finished dims of a query row from their sums, the maximum (log2 units) and the
// sum of the weights.
template <int DH>
__device__ __forceinline__ void kv4_rows_store(const Kv4AttnArgs &p, int b, int h, int row, int c4, float4 o, float m,
                                               float l) {
    if (row >= p.n_q) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;                 // no key: 0
    bf16 *dst = (bf16 *)p.out + ((int64_t)b * p.n_q + row) * ((int64_t)p.c.H * DH) + h * DH + c4;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (p.lse && c4 == 0)
        p.lse[((int64_t)h * p.B + b) * p.n_q + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * KV4_LN2;
}

// grid (query tiles of 8 NT rows, H, B * n_split), clusters of n_split CTAs where p.cluster
template <int DH, int NT>
__global__ void __launch_bounds__(32 * KV4R_WARPS, NT == 1 ? 3 : 2) k_kv4_attn_rows(const __grid_constant__ Kv4AttnArgs p) {
    using namespace sm100;
    using C = Kv4RowsCfg<DH, true>;
    constexpr int MT = DH / 16;                    // product tiles of 16 dims
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + KV4R_WARPS * C::STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (threadIdx.x == 0) {
        for (int i = 0; i < KV4R_WARPS * C::STAGES; ++i) mbar_init(smem_u32(&bars[i]), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.y, b = blockIdx.z / p.n_split, sp = blockIdx.z - b * p.n_split, cb = p.shared ? 0 : b;
    const int q0 = blockIdx.x * 8 * NT;
    const int64_t d = (int64_t)p.c.H * DH;
    const int len = kv4_len(p.c, p.prefix_len, cb);
    const int cp = (len + KV4R_CHUNK - 1) / KV4R_CHUNK, ct = (p.n_tail + KV4R_CHUNK - 1) / KV4R_CHUNK;
    const int lo = (int)((int64_t)sp * (cp + ct) / p.n_split), hi = (int)((int64_t)(sp + 1) * (cp + ct) / p.n_split);
    // this warp's chunks: lo + warp, lo + warp + 4, ..; the first n_pre of them prefix chunks
    const int first = lo + warp;
    const int n_all = first < hi ? (hi - first + KV4R_WARPS - 1) / KV4R_WARPS : 0;
    const int n_pre = first < min(hi, cp) ? (min(hi, cp) - first + KV4R_WARPS - 1) / KV4R_WARPS : 0;
    Kv4Ring<DH, true> ring;
    ring.stages = smem + warp * C::STAGES * C::STAGE;
    ring.bars = bars + warp * C::STAGES;
    const int64_t kr = kv4_row0(p.c, p.layer, 0, cb, h), vr = kv4_row0(p.c, p.layer, 1, cb, h);
    ring.k_codes = p.base + kr * (DH / 2);
    ring.v_codes = p.base + vr * (DH / 2);
    ring.k_scales = p.base + p.c.scales_off + kr * (C::G * 2);
    ring.v_scales = p.base + p.c.scales_off + vr * (C::G * 2);
    if (lane == 0)
        for (int n = 0; n < min(n_pre, C::STAGES); ++n) ring.load(n, first + n * KV4R_WARPS);
    uint32_t bq[NT][DH / 16][2];
    kv4_load_q<DH, NT>((const bf16 *)p.q + (int64_t)b * p.n_q * d + h * DH, q0, p.n_q, d, g, t, bq);
    const bf16 *kt = (const bf16 *)p.k_tail + (int64_t)b * p.n_tail * d + h * DH;
    const bf16 *vt = (const bf16 *)p.v_tail + (int64_t)b * p.n_tail * d + h * DH;

    float o[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[m][j][i] = 0.f;
    // queries 2t and 2t + 1 of each tile; l is this thread's keys only until the end
    float mr[NT][2], lr[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) mr[j][0] = mr[j][1] = -INFINITY, lr[j][0] = lr[j][1] = 0.f;

    for (int n = 0; n < n_all; ++n) {
        const int chunk = first + n * KV4R_WARPS;
        const bool pre = n < n_pre;
        const int n_keys = pre ? len - chunk * KV4R_CHUNK : p.n_tail - (chunk - cp) * KV4R_CHUNK;
        const uint8_t *st = ring.stages + (n % C::STAGES) * C::STAGE;
        const bf16 *kc = kt + (int64_t)(chunk - cp) * KV4R_CHUNK * d, *vc = vt + (int64_t)(chunk - cp) * KV4R_CHUNK * d;
        if (pre) {
            const bool ok = mbar_wait_settled(smem_u32(&ring.bars[n % C::STAGES]), (n / C::STAGES) & 1, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok ? 1 : 0)) break;
        }
        float s[KV4R_M][NT][4];
        if (pre) {
#pragma unroll
            for (int m = 0; m < KV4R_M; m += 2)
                kv4_scores_staged<DH, NT, 2>(st, st + C::CODES, 16 * m, g, t, bq, p.lop, s + m);
        } else {
#pragma unroll
            for (int m = 0; m < KV4R_M; ++m) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[m][j][i] = 0.f;
#pragma unroll
                for (int w = 0; w < DH / 32; ++w) {
                    uint4 ua = make_uint4(0, 0, 0, 0), ub = ua;
                    const bf16 *pa = kc + (int64_t)(16 * m + g) * d + t * (DH / 4) + w * 8;
                    if (16 * m + g < n_keys) ua = *reinterpret_cast<const uint4 *>(pa);
                    if (16 * m + g + 8 < n_keys) ub = *reinterpret_cast<const uint4 *>(pa + 8 * d);
                    uint32_t ka[4], kb[4];
                    kv4_order(ua, ka);
                    kv4_order(ub, kb);
                    kv4_scores_step<DH, NT>(ka, kb, w, bq, s[m]);
                }
            }
        }
        // softmax of the chunk: scores of keys 16 m + g (values 0, 1) and 16 m + 8 + g (2, 3)
        const bool partial = n_keys < KV4R_CHUNK;
        if (partial) {
#pragma unroll
            for (int m = 0; m < KV4R_M; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (16 * m + g + (i >> 1) * 8 >= n_keys) s[m][j][i] = -INFINITY;
        }
        bool moved = false;
        float alpha[NT][2], mc[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float mx = mr[j][i];
#pragma unroll
                for (int m = 0; m < KV4R_M; ++m) mx = fmax3(mx, s[m][j][i], s[m][j][i + 2]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                mc[j][i] = mx == -INFINITY ? 0.f : mx * p.scale_log2;
                alpha[j][i] = ex2_approx(fmaf(mr[j][i], p.scale_log2, -mc[j][i]));
                moved |= mx != mr[j][i];
                mr[j][i] = mx;
            }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int m = 0; m < KV4R_M; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[m][j][i] = ex2_approx(fmaf(s[m][j][i], p.scale_log2, -mc[j][i & 1]));
                    sum[i & 1] += s[m][j][i];
                }
            lr[j][0] = fmaf(lr[j][0], alpha[j][0], sum[0]);
            lr[j][1] = fmaf(lr[j][1], alpha[j][1], sum[1]);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[m][j][0] *= alpha[j][0];
                    o[m][j][1] *= alpha[j][1];
                    o[m][j][2] *= alpha[j][0];
                    o[m][j][3] *= alpha[j][1];
                }
        }
        // O^T += V^T P^T, 16 keys at a time
#pragma unroll
        for (int m = 0; m < KV4R_M; ++m) {
            uint32_t bp[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                bp[j][0] = movmatrix_trans(pack_bf16x2(s[m][j][0], s[m][j][1]));
                bp[j][1] = movmatrix_trans(pack_bf16x2(s[m][j][2], s[m][j][3]));
            }
            uint32_t a[4][MT];                     // operand register r of product tile i: a[r][i]
            if (pre) {
                const uint8_t *vcodes = st + C::CODES + C::SCALES, *vscales = vcodes + C::CODES;
#pragma unroll
                for (int half = 0; half < 2; ++half) {        // keys 2t, 2t + 1 and 8 more
                    const int k0 = 16 * m + 8 * half + 2 * t;
                    const int grp = g * C::G / 8;
                    uint32_t s0 = *reinterpret_cast<const uint16_t *>(vscales + (k0 * C::G + grp) * 2);
                    uint32_t s1 = *reinterpret_cast<const uint16_t *>(vscales + ((k0 + 1) * C::G + grp) * 2);
                    if (partial) {                             // what rows that do not exist hold stays out
                        if (k0 >= n_keys) s0 = 0;
                        if (k0 + 1 >= n_keys) s1 = 0;
                    }
                    const uint32_t s2 = __byte_perm(s0, s1, 0x5410), o2 = kv4_offset_pair(s2);
                    const uint8_t *pv = vcodes + k0 * (DH / 2) + g * (DH / 16);
                    if (DH == 128) {
                        const uint2 w0 = *reinterpret_cast<const uint2 *>(pv);
                        const uint2 w1 = *reinterpret_cast<const uint2 *>(pv + DH / 2);
                        uint32_t x[4];
                        kv4_pairs(__byte_perm(w0.x, w1.x, 0x5410), s2, o2, p.lop, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[2 * half][i] = x[i];
                        kv4_pairs(__byte_perm(w0.x, w1.x, 0x7632), s2, o2, p.lop, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[2 * half][(MT - 4) + i] = x[i];
                        kv4_pairs(__byte_perm(w0.y, w1.y, 0x5410), s2, o2, p.lop, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[2 * half + 1][i] = x[i];
                        kv4_pairs(__byte_perm(w0.y, w1.y, 0x7632), s2, o2, p.lop, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[2 * half + 1][(MT - 4) + i] = x[i];
                    } else {
                        const uint32_t w0 = *reinterpret_cast<const uint32_t *>(pv);
                        const uint32_t w1 = *reinterpret_cast<const uint32_t *>(pv + DH / 2);
                        uint32_t x[4];
                        kv4_pairs(__byte_perm(w0, w1, 0x5410), s2, o2, p.lop, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[2 * half][i] = x[i];
                        kv4_pairs(__byte_perm(w0, w1, 0x7632), s2, o2, p.lop, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[2 * half + 1][i] = x[i];
                    }
                }
            } else {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int k0 = 16 * m + 8 * half + 2 * t;
                    const bf16 *pv = vc + (int64_t)k0 * d + g * (DH / 8);
#pragma unroll
                    for (int w = 0; w < DH / 64; ++w) {        // 8 dims of both keys
                        uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
                        if (k0 < n_keys) u0 = *reinterpret_cast<const uint4 *>(pv + w * 8);
                        if (k0 + 1 < n_keys) u1 = *reinterpret_cast<const uint4 *>(pv + d + w * 8);
                        const uint32_t e0[4] = {u0.x, u0.y, u0.z, u0.w}, e1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {          // dim 8 w + i of the thread's
                            const uint32_t v = __byte_perm(e0[i >> 1], e1[i >> 1], i & 1 ? 0x7632 : 0x5410);
                            if (DH == 128) a[2 * half + w][i % MT] = v;
                            else a[2 * half + (i >> 2)][i & 3] = v;
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) mma_bf16(o[i][j], a[0][i], a[1][i], a[2][i], a[3][i], bp[j][0], bp[j][1]);
        }
        __syncwarp();
        if (pre && lane == 0 && n + C::STAGES < n_pre) ring.load(n + C::STAGES, chunk + C::STAGES * KV4R_WARPS);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) lr[j][i] += __shfl_xor_sync(0xffffffffu, lr[j][i], x);

    // merge the warps: [warp][m, l][8 NT] and [warp][8 NT][DH] floats, over the rings
    __syncthreads();
    float *st_m = reinterpret_cast<float *>(smem), *st_o = st_m + KV4R_WARPS * 2 * 8 * NT;
    if (g == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                st_m[(warp * 2 + 0) * 8 * NT + 8 * j + 2 * t + i] = mr[j][i] * p.scale_log2;
                st_m[(warp * 2 + 1) * 8 * NT + 8 * j + 2 * t + i] = lr[j][i];
            }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // rows g and g + 8 of product tile m: dims g Dh/8 + m, and half of Dh/8 further
                const int dim = g * (DH / 8) + (i >> 1) * (DH / 16) + m;
                st_o[(warp * 8 * NT + 8 * j + 2 * t + (i & 1)) * DH + dim] = o[m][j][i];
            }
    __syncthreads();
    // the CTA's own result, not normalised: a thread keeps its elements of it
    constexpr int ELEMS = 8 * NT * (DH / 4), PER = (ELEMS + 32 * KV4R_WARPS - 1) / (32 * KV4R_WARPS);
    float4 acc[PER];
    float am[PER], al[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * 32 * KV4R_WARPS, r = e / (DH / 4), c4 = (e - r * (DH / 4)) * 4;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < KV4R_WARPS; ++w) m = fmaxf(m, st_m[w * 2 * 8 * NT + r]);
        const float mz = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        float4 v4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KV4R_WARPS; ++w) {
            const float f = ex2_approx(st_m[w * 2 * 8 * NT + r] - mz);
            l = fmaf(f, st_m[(w * 2 + 1) * 8 * NT + r], l);
            const float4 v = *reinterpret_cast<const float4 *>(st_o + (w * 8 * NT + r) * DH + c4);
            v4.x = fmaf(f, v.x, v4.x);
            v4.y = fmaf(f, v.y, v4.y);
            v4.z = fmaf(f, v.z, v4.z);
            v4.w = fmaf(f, v.w, v4.w);
        }
        acc[i] = v4;
        am[i] = m;
        al[i] = l;
    }
    if (p.cluster) {
        // the splits are the CTAs of a cluster: every one publishes its result and
        // finishes a share of the elements from all of them
        __syncthreads();
        float *cl = reinterpret_cast<float *>(smem);            // [ELEMS] x (4 outputs, m, l)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x + i * 32 * KV4R_WARPS;
            if (e < ELEMS) {
                reinterpret_cast<float4 *>(cl)[e] = acc[i];
                reinterpret_cast<float2 *>(cl + 4 * ELEMS)[e] = make_float2(am[i], al[i]);
            }
        }
        cluster_sync();
        const uint32_t base = smem_u32(cl);
        for (int e = sp * 32 * KV4R_WARPS + threadIdx.x; e < ELEMS; e += p.n_split * 32 * KV4R_WARPS) {
            float m = -INFINITY;
            float2 ml[KV4R_CLUSTER];
            float4 v[KV4R_CLUSTER];
#pragma unroll
            for (int w = 0; w < KV4R_CLUSTER; ++w) {
                ml[w] = make_float2(-INFINITY, 0.f);
                v[w] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (w < p.n_split) {
                    ml[w] = ld_cluster_f2(mapa_shared(base + 16 * ELEMS + 8 * e, w));
                    v[w] = ld_cluster_f4(mapa_shared(base + 16 * e, w));
                    m = fmaxf(m, ml[w].x);
                }
            }
            const float mz = m == -INFINITY ? 0.f : m;
            float l = 0.f;
            float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < KV4R_CLUSTER; ++w) {
                const float f = ex2_approx(ml[w].x - mz);
                l = fmaf(f, ml[w].y, l);
                o4.x = fmaf(f, v[w].x, o4.x);
                o4.y = fmaf(f, v[w].y, o4.y);
                o4.z = fmaf(f, v[w].z, o4.z);
                o4.w = fmaf(f, v[w].w, o4.w);
            }
            kv4_rows_store<DH>(p, b, h, q0 + e / (DH / 4), (e % (DH / 4)) * 4, o4, m, l);
        }
        cluster_sync();                                        // nobody leaves while it is read
        return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * 32 * KV4R_WARPS, r = e / (DH / 4), c4 = (e - r * (DH / 4)) * 4, row = q0 + r;
        if (e >= ELEMS || row >= p.n_q) continue;
        if (p.n_split == 1) {
            kv4_rows_store<DH>(p, b, h, row, c4, acc[i], am[i], al[i]);
        } else {
            const float inv = al[i] == 0.f ? 0.f : 1.f / al[i];
            const int64_t at = (((int64_t)b * p.c.H + h) * p.n_split + sp) * p.n_q + row;
            *reinterpret_cast<float4 *>(p.part_o + at * DH + c4) =
                make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
            if (c4 == 0) p.part_l[at] = al[i] == 0.f ? -INFINITY : am[i] + log2f(al[i]);
        }
    }
}

// The weights of a few query rows: the same stream over K alone. Queries in passes of
// 8 NT over the staged chunk. grid (key splits, H, cache items); a split's warps take
// its chunks in turn, and every key's sum is one warp's.
template <int DH>
__global__ void __launch_bounds__(32 * KV4R_WARPS, 4) k_kv4_scores_rows(const __grid_constant__ Kv4ScoreArgs p) {
    using namespace sm100;
    using C = Kv4RowsCfg<DH, false>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + KV4R_WARPS * C::STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (threadIdx.x == 0) {
        for (int i = 0; i < KV4R_WARPS * C::STAGES; ++i) mbar_init(smem_u32(&bars[i]), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.y, b = blockIdx.z;
    const int64_t d = (int64_t)p.c.H * DH;
    const int len = kv4_len(p.c, p.prefix_len, b);
    const float *in = p.in ? p.in + ((int64_t)b * p.c.H + h) * p.c.P : nullptr;
    float *out = p.out + ((int64_t)b * p.c.H + h) * p.c.P;
    const int chunks = (p.c.P + KV4R_CHUNK - 1) / KV4R_CHUNK;
    const int lo = (int)((int64_t)blockIdx.x * chunks / gridDim.x), hi = (int)((int64_t)(blockIdx.x + 1) * chunks / gridDim.x);
    const int first = lo + warp;
    const int n_all = first < hi ? (hi - first + KV4R_WARPS - 1) / KV4R_WARPS : 0;
    const int end = min(hi, (len + KV4R_CHUNK - 1) / KV4R_CHUNK);
    const int n_pre = first < end ? (end - first + KV4R_WARPS - 1) / KV4R_WARPS : 0;
    Kv4Ring<DH, false> ring;
    ring.stages = smem + warp * C::STAGES * C::STAGE;
    ring.bars = bars + warp * C::STAGES;
    const int64_t kr = kv4_row0(p.c, p.layer, 0, b, h);
    ring.k_codes = p.base + kr * (DH / 2);
    ring.k_scales = p.base + p.c.scales_off + kr * (C::G * 2);
    ring.v_codes = ring.v_scales = nullptr;
    if (lane == 0)
        for (int n = 0; n < min(n_pre, C::STAGES); ++n) ring.load(n, first + n * KV4R_WARPS);
    const bf16 *q = (const bf16 *)p.q + (int64_t)b * p.n_q * d + h * DH;
    const float *lse = p.lse + ((int64_t)h * p.c.B + b) * p.n_q;
    uint32_t bq[1][DH / 16][2];
    float off[2];
    auto fetch = [&](int q0) {
        kv4_load_q<DH, 1>(q, q0, p.n_q, d, g, t, bq);
#pragma unroll
        for (int i = 0; i < 2; ++i) off[i] = q0 + 2 * t + i < p.n_q ? -kv4_lse2(lse[q0 + 2 * t + i]) : -INFINITY;
    };
    fetch(0);
    for (int n = 0; n < n_all; ++n) {
        const int chunk = first + n * KV4R_WARPS, n_keys = n < n_pre ? len - chunk * KV4R_CHUNK : 0;
        float sum[KV4R_M][2];                               // keys 16 m + g and 16 m + 8 + g
#pragma unroll
        for (int m = 0; m < KV4R_M; ++m) sum[m][0] = sum[m][1] = 0.f;
        if (n < n_pre) {
            const uint8_t *st = ring.stages + (n % C::STAGES) * C::STAGE;
            const bool ok = mbar_wait_settled(smem_u32(&ring.bars[n % C::STAGES]), (n / C::STAGES) & 1, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok ? 1 : 0)) break;
            for (int q0 = 0; q0 < p.n_q; q0 += 8) {
                if (p.n_q > 8) fetch(q0);
                float s[KV4R_M][1][4];
#pragma unroll
                for (int m = 0; m < KV4R_M; ++m)
                    kv4_scores_staged<DH, 1, 1, true>(st, st + C::CODES, 16 * m, g, t, bq, p.lop, s + m);
#pragma unroll
                for (int m = 0; m < KV4R_M; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sum[m][i >> 1] += ex2_approx(fmaf(s[m][0][i], p.scale_log2, off[i & 1]));
            }
            __syncwarp();
            if (lane == 0 && n + C::STAGES < n_pre) ring.load(n + C::STAGES, chunk + C::STAGES * KV4R_WARPS);
        }
#pragma unroll
        for (int m = 0; m < KV4R_M; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float a = sum[m][i];
                a += __shfl_xor_sync(0xffffffffu, a, 1);
                a += __shfl_xor_sync(0xffffffffu, a, 2);
                const int r = 16 * m + 8 * i + g, j = chunk * KV4R_CHUNK + r;
                if (t == 0 && j < p.c.P && (r < n_keys || out != in)) out[j] = (in ? in[j] : 0.f) + (r < n_keys ? a : 0.f);
            }
    }
}

}  // namespace qi21
