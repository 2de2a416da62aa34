// Prefix K/V cache held in 4 bits: the format, the kernels that write it, read
// it back and evict rows from it, and the CUDA-core forms of the attention over
// it and of the accumulated attention weight (the F32 mode).
//
// Format. A group is 32 consecutive dims of one head of one row. With
// a = max |x| of the group, its scale s is 0 if a = 0, else the smallest number
// with a 5-bit significand for which 7 s >= a (kept in [2^-126, 2^122], held as
// bf16); an element is k = rint(x / s), ties to even, in [-7, 7], stored as k + 8
// in 4 bits. k has at most 3 significant bits and s has 5, so the value k s has
// at most 8: it is exact in bf16, and every kernel multiplies the same numbers
// whether it works in bf16 or in fp32. The rounding to k is the only loss.
// 4 + 16/32 = 4.5 bits an element.
//
// Layout (one buffer): codes [L][K|V][B][H][Pp][Dh/2] bytes (dim 2i in the low
// half of byte i), then scales [L][K|V][B][H][Pp][Dh/32] bf16; Pp = P rounded up
// to the 128-key tile. Head-major, so that the rows an attention CTA reads are
// contiguous; every row carries its own scales, so that evicting rows is a plain
// gather. Rows [P, Pp) are never written, and no kernel lets what they (or the
// rows behind an item's own length) hold reach a result.
#pragma once
#include "qi21_attn_tc.cuh"     // packed fp32 pairs
#include "qi21_common.cuh"

namespace qi21 {

constexpr int KV4_GROUP = 32;

struct Kv4Dims {
    int B, H, P, Pp, Dh;
    int64_t scales_off;          // bytes from the buffer's start to the scales
};

__host__ __device__ __forceinline__ int64_t kv4_pad(int64_t P) { return (P + 127) / 128 * 128; }

// First row of (layer l, which = 0 K / 1 V, item b, head h), in rows.
__host__ __device__ __forceinline__ int64_t kv4_row0(const Kv4Dims &c, int l, int which, int b, int h) {
    return ((((int64_t)l * 2 + which) * c.B + b) * c.H + h) * c.Pp;
}

// Rows of item b that exist: its own length where the cache has lengths, else P.
__device__ __forceinline__ int kv4_len(const Kv4Dims &c, const int *prefix_len, int b) {
    if (!prefix_len) return c.P;
    const int n = prefix_len[b];
    return n < 0 ? 0 : (n > c.P ? c.P : n);
}

// ------------------------------------------------------------------ expanding codes
// The two constants of the expansion to bf16 (kv4_pairs), as kernel parameters: from
// there both are register or constant-bank operands and (w & mask) | one is a single
// LOP3; as literals they are two.
struct Kv4Lop {
    uint32_t mask, one;          // 0x00780078, 0x41804180
};
constexpr Kv4Lop kKv4Lop{0x00780078u, 0x41804180u};

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t kv4_scale_pair(uint32_t s) {
    uint32_t p;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(p) : "r"(s));
    return p;
}
__device__ __forceinline__ uint32_t kv4_offset_pair(uint32_t s2) {   // -24 s, exact
    return fma_bf16x2(s2, 0xC1C0C1C0u, 0x80008000u);
}
// Nibbles i and i + 4 of w, i = 0 .. 3, as the values of a pair.
__device__ __forceinline__ uint32_t kv4_nibbles(uint32_t w, const Kv4Lop &k) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(k.mask), "r"(k.one));   // (w & mask) | one
    return d;
}
// (nibble - 8) s of the 8 nibbles of a code word as bf16 pairs: in the order in which it
// unfolds (nibbles i and i + 4), and in the order of dims.
__device__ __forceinline__ void kv4_pairs(uint32_t w, uint32_t s2, uint32_t off2, const Kv4Lop &k, uint32_t (&p)[4]) {
    p[0] = fma_bf16x2(kv4_nibbles(w << 3, k), s2, off2);
    p[1] = fma_bf16x2(kv4_nibbles(w >> 1, k), s2, off2);
    p[2] = fma_bf16x2(kv4_nibbles(w >> 5, k), s2, off2);
    p[3] = fma_bf16x2(kv4_nibbles(w >> 9, k), s2, off2);
}
__device__ __forceinline__ uint4 kv4_expand(uint32_t w, uint32_t s2, uint32_t off2, const Kv4Lop &k) {
    uint32_t p[4];
    kv4_pairs(w, s2, off2, k, p);
    return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                      __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632));
}

// ------------------------------------------------------------------ quantise
// 8 consecutive elements of a row as floats.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16 *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The scale of a group whose largest magnitude has these bits (finite or not).
// The candidate cuts a/7 (a product with the rounded 1/7, within 2^-23 of it) to
// 5 bits; one step up where 7 times it falls short. 7 * (5 bits) is exact in
// fp32, so the test is exact. A NaN or an infinity anywhere makes the scale NaN.
__device__ __forceinline__ float kv4_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    const float a = __uint_as_float(amax_bits);
    if (a == 0.f) return 0.f;
    constexpr float lo = 1.17549435e-38f, hi = 5.316911983e36f;   // 2^-126, 2^122
    float s = __uint_as_float(__float_as_uint(a * 0.142857149f) & 0xFFF80000u);
    if (s < lo) s = lo;      // below the smallest normal number there are not 5 bits
    if (7.f * s < a) s = __uint_as_float(__float_as_uint(s) + 0x00080000u);
    return fminf(s, hi);
}

// The code word of 8 elements of a group with scale s > 0: rint(x / s), ties to even,
// in [-7, 7], plus 8. With r = 1 / s (within 2^-22) and M = 1.5 2^23 + 8 the two sums
// x r (1 + 2^-20) + M and x r (1 - 2^-20) + M, each rounded once, hold integers k+ + 8
// and k- + 8 in their low bits; where they are equal, that is the nearest integer to
// the quotient, which lies between them. Their own sum has a unit of 2, so that it is
// rounded to the even one of k+ and k- where these differ: the tie rule. For bf16
// elements they differ at ties alone (8 bits over 5: a quotient that is not a half
// integer is at least 1/1984 away from one). Elements of 24 bits can be nearer; there
// the remainder x - k s decides, which is exact (k s has 8 bits, and the difference
// is x itself or exact by Sterbenz' lemma).
template <bool EXACT>
__device__ __forceinline__ uint32_t kv4_code_word(const float (&x)[8], float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    const float up = r * (1.f + 0x1p-20f), dn = r * (1.f - 0x1p-20f), M = 12582920.f;
    uint32_t b[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {               // packed pairs
        const uint64_t v = f2_pack(x[k], x[k + 1]);
        const uint64_t a2 = f2_fma(v, f2_pack(up, up), f2_pack(M, M)), c2 = f2_fma(v, f2_pack(dn, dn), f2_pack(M, M));
        float a[2], c[2], t[2];
        f2_unpack(f2_add(a2, c2), t[0], t[1]);
        f2_unpack(a2, a[0], a[1]);
        f2_unpack(c2, c[0], c[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            b[k + i] = __float_as_uint(t[i]);
            if (EXACT && a[i] != c[i]) {
                float q = fminf(a[i], c[i]) - M;           // the lower of the two integers
                const float e = fmaf(-q, s, x[k + i]), h = 0.5f * s;
                if (e > h || (e == h && ((int)q & 1))) q += 1.f;
                b[k + i] = __float_as_uint(2.f * (q + M));
            }
        }
    }
    // the low bytes hold the codes: even ones, and odd ones a nibble further
    const uint32_t e = __byte_perm(__byte_perm(b[0], b[2], 0x0040), __byte_perm(b[4], b[6], 0x0040), 0x5410);
    const uint32_t o = __byte_perm(__byte_perm(b[1], b[3], 0x0040), __byte_perm(b[5], b[7], 0x0040), 0x5410);
    return e + 16u * o;
}

// 8 consecutive elements as they are stored: the bits (of a float) of the largest
// magnitude, where a NaN's lie above all others, and the elements as floats.
template <typename T> struct Kv4Row8;
template <> struct Kv4Row8<float> {
    float x[8];
    __device__ __forceinline__ void load(const float *p) { load8(p, x); }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0.f;
    }
    __device__ __forceinline__ uint32_t max_bits() const {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7FFFFFFFu);
        return m;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = x[k];
    }
};
template <> struct Kv4Row8<bf16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const bf16 *p) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    }
    __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ uint32_t max_bits() const {       // both halves of a word at once
        uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int k = 1; k < 4; ++k) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k] & 0x7FFF7FFFu));
        return max(m & 0xFFFF0000u, m << 16);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    }
};

constexpr int KV4_Q_ROWS = 2;    // rows of one column that a thread of the quantiser handles
constexpr int KV4_D_ROWS = 4;    // and of the way back

// Quantise rows [0, P) of every (layer, K|V, item) slab of a cache in token-major
// layout (slab stride in elements) into the 4-bit layout. A thread takes 16
// consecutive dims of two consecutive rows; the two threads of a group share its
// maximum by a shuffle. Bound by HBM (eb + 0.5625 bytes an element) and the issue
// slots alike (some 6 operations an element): 120 us for 277 M elements of bf16 (5.9
// TB/s; 139 us with 8 dims a thread, whose scale costs as much).
template <typename T>
__global__ void __launch_bounds__(256) k_kv4_quantize(const T *src, int64_t slab_stride, Kv4Dims c,
                                                      const int *prefix_len, uint8_t *base) {
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t d = c.H * c.Dh, cols = d / 16, u = blockIdx.x * 256 + threadIdx.x;
    const int slab = blockIdx.y;                 // (l * 2 + which) * B + b
    const int rows = kv4_len(c, prefix_len, slab % c.B);
    const uint32_t pair = u / cols, col = u - pair * cols;   // the 2 threads of a group share a warp: cols % 2 == 0
    const uint32_t h = col * 16 / c.Dh, j0 = col * 16 - h * c.Dh;
    const int64_t r0 = (int64_t)pair * KV4_Q_ROWS;
    const T *from = src + slab * slab_stride + r0 * d + col * 16;
    Kv4Row8<T> x[KV4_Q_ROWS][2];
#pragma unroll
    for (int i = 0; i < KV4_Q_ROWS; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (r0 + i < rows) x[i][k].load(from + i * d + k * 8);
            else x[i][k].zero();
        }
    const int64_t row0 = ((int64_t)slab * c.H + h) * c.Pp + r0;
    const uint32_t row_codes = c.Dh / 2, row_scales = c.Dh / KV4_GROUP;
    uint8_t *codes = base + row0 * row_codes + j0 / 2;
    uint16_t *scales = reinterpret_cast<uint16_t *>(base + c.scales_off) + row0 * row_scales + j0 / KV4_GROUP;
#pragma unroll
    for (int i = 0; i < KV4_Q_ROWS; ++i) {
        uint32_t m = max(x[i][0].max_bits(), x[i][1].max_bits());
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const float s = kv4_scale(m);
        const bool huge = __any_sync(0xffffffffu, m > 0x7DE00000u);     // beyond 7 * 2^122: saturate
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float v[8];
            x[i][k].get(v);
            if (huge) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fminf(fmaxf(v[e], -7.f * s), 7.f * s);
            }
            w[k] = kv4_code_word<sizeof(T) == 4>(v, s);
            if (!(s > 0.f)) w[k] = 0x88888888u;              // an empty group, or one that is not finite
        }
        if (r0 + i < rows) {
            *reinterpret_cast<uint2 *>(codes + i * row_codes) = make_uint2(w[0], w[1]);
            if ((col & 1) == 0) scales[i * row_scales] = (uint16_t)(__float_as_uint(s) >> 16);
        }
    }
}

// ------------------------------------------------------------------ dequantise
// The 8 values of a code word in each storage type.
__device__ __forceinline__ void kv4_store8(bf16 *p, uint32_t w, uint32_t s, const Kv4Lop &k) {
    const uint32_t s2 = kv4_scale_pair(s);
    *reinterpret_cast<uint4 *>(p) = kv4_expand(w, s2, kv4_offset_pair(s2), k);
}
__device__ __forceinline__ void kv4_store8(float *p, uint32_t w, uint32_t s, const Kv4Lop &k) {
    const uint32_t s2 = kv4_scale_pair(s);
    const uint4 v = kv4_expand(w, s2, kv4_offset_pair(s2), k);
    const uint32_t e[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(e[i] << 16);
        x[2 * i + 1] = __uint_as_float(e[i] & 0xFFFF0000u);
    }
    store8(p, x);
}
__device__ __forceinline__ void kv4_values(uint32_t w, float s, float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = (float)((int)((w >> (4 * k)) & 15u) - 8) * s;
}
__device__ __forceinline__ float kv4_load_scale(const uint8_t *base, const Kv4Dims &c, int64_t row, int group) {
    return __uint_as_float(
        (uint32_t)reinterpret_cast<const uint16_t *>(base + c.scales_off)[row * (c.Dh / KV4_GROUP) + group] << 16);
}

// The way back: rows [0, len) of slabs slab0, slab0 + 1, .. in token-major layout,
// 8 dims of four rows a thread. pad: zeros behind them up to a multiple of 128 rows
// (the tiles of an attention that reads the result). Bound by HBM: 112 us for 277 M
// elements to bf16 (6.3 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) k_kv4_dequantize(const uint8_t *base, Kv4Dims c, int slab0,
                                                        const int *prefix_len, int pad,
                                                        T *dst, int64_t slab_stride, Kv4Lop lop) {
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t d = c.H * c.Dh, cols = d / 8, u = blockIdx.x * 256 + threadIdx.x;
    const int slab = slab0 + blockIdx.y;
    const int rows = kv4_len(c, prefix_len, slab % c.B);
    const uint32_t quad = u / cols, col = u - quad * cols;
    const uint32_t h = col * 8 / c.Dh, j0 = col * 8 - h * c.Dh;
    const int64_t r0 = (int64_t)quad * KV4_D_ROWS, row0 = ((int64_t)slab * c.H + h) * c.Pp + r0;
    const uint8_t *codes = base + row0 * (c.Dh / 2) + j0 / 2;
    const uint16_t *scales =
        reinterpret_cast<const uint16_t *>(base + c.scales_off) + row0 * (c.Dh / KV4_GROUP) + j0 / KV4_GROUP;
    const int64_t rows_out = pad ? kv4_pad(rows) : rows;
    uint32_t w[KV4_D_ROWS], s[KV4_D_ROWS];
#pragma unroll
    for (int i = 0; i < KV4_D_ROWS; ++i) {
        w[i] = s[i] = 0;                         // the value 0
        if (r0 + i < rows) {
            w[i] = *reinterpret_cast<const uint32_t *>(codes + (int64_t)i * (c.Dh / 2));
            s[i] = scales[(int64_t)i * (c.Dh / KV4_GROUP)];
        }
    }
    T *to = dst + (int64_t)blockIdx.y * slab_stride + r0 * d + col * 8;
#pragma unroll
    for (int i = 0; i < KV4_D_ROWS; ++i)
        if (r0 + i < rows_out) kv4_store8(to + (int64_t)i * d, w[i], s[i], lop);
}

// ------------------------------------------------------------------ eviction
// Order of the eviction: protected rows first, then by score; a NaN score counts
// as the lowest of all.
__device__ __forceinline__ uint32_t kv4_rank(float s, int j, int n_protected) {
    if (j < n_protected) return 0xFFFFFFFFu;
    if (s != s) return 0u;
    const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);       // -0 ranks as +0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}


constexpr int KV4_GATHER = 4;    // rows of a thread

// Copy rows of K and V into the smaller cache: THREADS threads, those of the kept list
// from r0 on, four a thread. A thread moves one group (16 bytes of codes and its scale)
// of its rows, all of them in flight at once. Bound by HBM's latency and its 64-byte
// pieces: 38 us for 170 MB (8 layers, 32 heads of 128, 2304 of 4608 rows).
template <int THREADS>
__device__ __forceinline__ void kv4_gather_rows(const uint8_t *src, const Kv4Dims &c, const int *list, int keep, int r0,
                                                int l, int b, int h, uint8_t *dst, const Kv4Dims &o) {
    const uint32_t G = c.Dh / KV4_GROUP, rows = THREADS / G;   // G threads a row, `rows` rows at a time
    const uint32_t t = threadIdx.x / G, g = threadIdx.x - t * G;
    if (t >= rows) return;                                     // THREADS is no multiple of 3
    int j[KV4_GATHER];
#pragma unroll
    for (int i = 0; i < KV4_GATHER; ++i) {
        const int r = r0 + t + i * rows;
        j[i] = r < keep ? list[r] : -1;
    }
    const uint16_t *from_s = reinterpret_cast<const uint16_t *>(src + c.scales_off);
    uint16_t *to_s = reinterpret_cast<uint16_t *>(dst + o.scales_off);
    uint4 code[2][KV4_GATHER];
    uint16_t scale[2][KV4_GATHER];
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int i = 0; i < KV4_GATHER; ++i)
            if (j[i] >= 0) {
                const int64_t from = (kv4_row0(c, l, which, b, h) + j[i]) * G + g;
                code[which][i] = reinterpret_cast<const uint4 *>(src)[from];
                scale[which][i] = from_s[from];
            }
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int i = 0; i < KV4_GATHER; ++i)
            if (j[i] >= 0) {
                const int64_t to = (kv4_row0(o, l, which, b, h) + r0 + t + i * rows) * G + g;
                reinterpret_cast<uint4 *>(dst)[to] = code[which][i];
                to_s[to] = scale[which][i];
            }
}

// The rows that one (layer, item, head) keeps: the `keep` largest of its ranks,
// ties to the lowest row, in ascending order; -1 behind them where the item has
// fewer rows. Radix selection, 8 bits a pass from the top, on integers: exact, and
// the same whatever the order of the atomics. A thread holds IPT consecutive rows,
// so that one scan over the block gives every row its place; where the rows are more
// than THREADS x IPT, they are read again tile by tile in each pass. Bound by latency
// (barriers and one read of the scores): 10 us for 1024 heads of 512 rows, 18 us for
// 256 of 4608. GATHER: the block then copies the rows it has chosen, which runs under the
// selections of the blocks beside it. grid (H, B, L).
template <int THREADS, int IPT, bool GATHER>
__global__ void __launch_bounds__(THREADS)
    k_kv4_select(const float *scores, Kv4Dims c, const int *prefix_len, int keep, int n_protected, int *kept,
                 int *dst_len, const uint8_t *src, uint8_t *dst, Kv4Dims o) {
    constexpr int W = THREADS / 32, TILE = THREADS * IPT;
    static_assert(TILE <= 8192, "two counts share 32 bits");
    __shared__ int hist[2][256];
    __shared__ int sel[2], warp_sums[W];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    for (int i = tid; i < 512; i += THREADS) hist[i >> 8][i & 255] = 0;
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.x, b = blockIdx.y, l = blockIdx.z;
    const int64_t lbh = ((int64_t)l * c.B + b) * c.H + h;
    const float *sc = scores + lbh * c.P;
    int *out = kept + lbh * keep;
    const int len = kv4_len(c, prefix_len, b), count = min(keep, len), tiles = (len + TILE - 1) / TILE;
    if (dst_len && l == 0 && h == 0 && tid == 0) dst_len[b] = count;
    uint32_t key[IPT];
    auto load = [&](int tile) {
#pragma unroll
        for (int i = 0; i < IPT; ++i) {
            const int j = tile * TILE + tid * IPT + i;
            key[i] = j < len ? kv4_rank(sc[j], j, n_protected) : 0u;
        }
    };
    if (tiles == 1) load(0);
    uint32_t prefix = 0;         // the bits of the count-th largest rank found so far
    int need = count;            // how many ranks with these bits are taken
    if (count < len) {
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            const uint32_t mask = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
            int *hs = hist[pass & 1];
            __syncthreads();                                   // hs is zero
            if (tiles == 1) {
#pragma unroll
                for (int i = 0; i < IPT; ++i)
                    if (tid * IPT + i < len && (key[i] & mask) == prefix) atomicAdd(&hs[(key[i] >> shift) & 255], 1);
            } else {
                // the order does not matter here: neighbours read neighbours, 8 loads in flight
                for (int j0 = tid; j0 < len; j0 += 8 * THREADS) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = j0 + i * THREADS < len ? sc[j0 + i * THREADS] : 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = j0 + i * THREADS;
                        const uint32_t r = kv4_rank(v[i], j, n_protected);
                        if (j < len && (r & mask) == prefix) atomicAdd(&hs[(r >> shift) & 255], 1);
                    }
                }
            }
            __syncthreads();
            if (wid == 0) {
                // 8 bins a lane, the largest ones first: the bin in which the count is reached
                int n[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    n[i] = hs[255 - (lane * 8 + i)];
                    sum += n[i];
                }
                int upto = sum;
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, upto, x);
                    if (lane >= x) upto += v;
                }
                int before = upto - sum;
                if (before < need && upto >= need) {           // one lane
                    int i = 0;
#pragma unroll
                    for (int k = 0; k < 7; ++k)
                        if (i == k && before + n[k] < need) {
                            before += n[k];
                            ++i;
                        }
                    sel[0] = 255 - (lane * 8 + i);
                    sel[1] = need - before;
                }
            } else {
                for (int i = tid - 32; i < 256; i += THREADS - 32) hist[(pass + 1) & 1][i] = 0;   // for the next pass
            }
            __syncthreads();
            prefix |= (uint32_t)sel[0] << shift;
            need = sel[1];
        }
    }
    // places: the larger ranks before a row, and as many of its ties as are taken
    int above0 = 0, ties0 = 0;
    for (int t = 0; t < tiles; ++t) {
        if (tiles > 1) load(t);
        const int j0 = t * TILE + tid * IPT;
        int above = 0, ties = 0;
#pragma unroll
        for (int i = 0; i < IPT; ++i) {
            if (j0 + i >= len) continue;
            if (count == len || key[i] > prefix) ++above;
            else if (key[i] == prefix) ++ties;
        }
        int mine = above | (ties << 16), upto = mine;          // at most 8192 of each in a tile
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, x);
            if (lane >= x) upto += v;
        }
        __syncthreads();
        if (lane == 31) warp_sums[wid] = upto;
        __syncthreads();
        int base = 0, all = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int n = warp_sums[i];
            if (i < wid) base += n;
            all += n;
        }
        base += upto - mine;
        int a = above0 + (base & 0xFFFF), q = ties0 + (base >> 16);
#pragma unroll
        for (int i = 0; i < IPT; ++i) {
            if (j0 + i >= len) continue;
            const bool tie = count < len && key[i] == prefix;
            const bool take = count == len || key[i] > prefix || (tie && q < need);
            if (take) out[a + min(q, need)] = j0 + i;
            if (tie) ++q;
            else if (take) ++a;
        }
        above0 += all & 0xFFFF;
        ties0 += all >> 16;
    }
    for (int i = count + tid; i < keep; i += THREADS) out[i] = -1;
    if (GATHER) {
        __syncthreads();                       // the list that the block has written
        const int step = KV4_GATHER * (THREADS / (c.Dh / KV4_GROUP));
        for (int r0 = 0; r0 < count; r0 += step) kv4_gather_rows<THREADS>(src, c, out, count, r0, l, b, h, dst, o);
    }
}

// The gather by itself, for few heads with many rows each. grid (blocks of rows, H, L * B).
static __global__ void __launch_bounds__(256)
    k_kv4_gather(const uint8_t *src, Kv4Dims c, const int *kept, int keep, uint8_t *dst, Kv4Dims o) {
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.y, l = blockIdx.z / c.B, b = blockIdx.z - l * c.B;
    kv4_gather_rows<256>(src, c, kept + (((int64_t)l * c.B + b) * c.H + h) * keep, keep,
                         blockIdx.x * (KV4_GATHER * (256 / (c.Dh / KV4_GROUP))), l, b, h, dst, o);
}

// ------------------------------------------------------------------ CUDA-core attention
// Keys of an item, in this order: its prefix rows [0, len) from the 4-bit cache,
// then its n_tail tail rows (token-major, storage dtype). 32 query rows x 32 keys
// a step, 128 threads: 2 x 4 scores a thread, then 4 rows x DH/16 dims of the
// output. fp32 throughout. The keys are split over n_split CTAs whose normalised
// partial outputs and log2-sum-exps k_kv4_combine joins. The F32 mode is the parity
// mode: 27 TFLOP/s at 8 x 256 rows, 768 keys, 16 heads of 64, bound by the loads of its
// tiles from shared memory.
struct Kv4AttnArgs {
    const uint8_t *base;
    Kv4Dims c;
    const int *prefix_len;
    int layer;
    int shared;                  // 1: every item reads cache item 0
    const void *q;               // [B][n_q][d]
    int B, n_q;
    const void *k_tail, *v_tail; // [B][n_tail][d]
    int n_tail;
    void *out;                   // [B][n_q][d]
    float *lse;                  // [H][B][n_q] or null
    int n_split, cluster;        // cluster: the splits are merged within a cluster
    float *part_l;               // [B][H][n_split][n_q]       log2-sum-exp
    float *part_o;               // [B][H][n_split][n_q][DH]
    float scale_log2;            // log2(e) / sqrt(Dh)
    uint32_t *err;
    Kv4Lop lop;
};

constexpr float KV4_LN2 = 0.69314718055994531f;

// Rows [r0, r0 + 32) of one head of a token-major tensor into shared memory, zeros behind n.
template <typename T, int DH>
__device__ __forceinline__ void kv4_stage_rows(float *dst, const T *src, int r0, int n, int d) {
    for (int e = threadIdx.x; e < 32 * (DH / 8); e += 128) {
        const int i = e / (DH / 8), c8 = e - i * (DH / 8);
        float x[8];
        if (r0 + i < n) {
            load8(src + (int64_t)(r0 + i) * d + c8 * 8, x);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = 0.f;
        }
        store8(dst + i * (DH + 4) + c8 * 8, x);
    }
}

// Keys [k0, k0 + 32) of an item (prefix, then tail), zeros from k_end on.
template <typename T, int DH>
__device__ __forceinline__ void kv4_stage_keys(float *dst, const uint8_t *base, const Kv4Dims &c, int64_t row0,
                                               int len, const T *tail, int d, int k0, int k_end) {
    for (int e = threadIdx.x; e < 32 * (DH / 8); e += 128) {
        const int i = e / (DH / 8), c8 = e - i * (DH / 8), key = k0 + i;
        float x[8];
        if (key < k_end && key < len) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(base + (row0 + key) * (DH / 2) + c8 * 4);
            kv4_values(w, kv4_load_scale(base, c, row0 + key, c8 / 4), x);
        } else if (key < k_end) {
            load8(tail + (int64_t)(key - len) * d + c8 * 8, x);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = 0.f;
        }
        store8(dst + i * (DH + 4) + c8 * 8, x);
    }
}

// acc[i][j] = A[2 ty + i] . B[tx + 8 j] over DH, both [32][DH + 4] in shared memory.
template <int DH>
__device__ __forceinline__ void kv4_tile_product(const float *A, const float *Bm, int ty, int tx, float (&acc)[2][4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < DH; k += 4) {
        float4 a[2], b[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = *reinterpret_cast<const float4 *>(A + (2 * ty + i) * (DH + 4) + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(Bm + (tx + 8 * j) * (DH + 4) + k);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
                acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
                acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
                acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
            }
    }
}

template <int DH>
constexpr size_t kv4_attn_simt_smem() {
    return sizeof(float) * (3 * 32 * (DH + 4) + 32 * 36 + 3 * 32);
}

// grid (query tiles, H, B * n_split)
template <typename T, int DH>
__global__ void __launch_bounds__(128) k_kv4_attn_simt(Kv4AttnArgs p) {
    extern __shared__ __align__(16) float sm4[];
    float *Qs = sm4, *Ks = Qs + 32 * (DH + 4), *Vs = Ks + 32 * (DH + 4);
    float *Ps = Vs + 32 * (DH + 4);          // [key][36]: row r of key k at k * 36 + r
    float *al = Ps + 32 * 36, *ls = al + 32, *ms = ls + 32;
    const int h = blockIdx.y, b = blockIdx.z / p.n_split, sp = blockIdx.z - b * p.n_split;
    const int q0 = blockIdx.x * 32, d = p.c.H * DH, cb = p.shared ? 0 : b;
    const int tid = threadIdx.x, ty = tid >> 3, tx = tid & 7, py = tid >> 4, px = tid & 15;
    const int len = kv4_len(p.c, p.prefix_len, cb), keys = len + p.n_tail;
    const int per = ((keys + p.n_split - 1) / p.n_split + 31) / 32 * 32;
    const int k_lo = min(keys, sp * per), k_hi = min(keys, k_lo + per);
    const int64_t k_row0 = kv4_row0(p.c, p.layer, 0, cb, h), v_row0 = kv4_row0(p.c, p.layer, 1, cb, h);
    const T *kt = (const T *)p.k_tail + (int64_t)b * p.n_tail * d + h * DH;
    const T *vt = (const T *)p.v_tail + (int64_t)b * p.n_tail * d + h * DH;
    kv4_stage_rows<T, DH>(Qs, (const T *)p.q + (int64_t)b * p.n_q * d + h * DH, q0, p.n_q, d);
    constexpr int NC = DH / 16;
    float o[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NC; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int k0 = k_lo; k0 < k_hi; k0 += 32) {
        __syncthreads();
        kv4_stage_keys<T, DH>(Ks, p.base, p.c, k_row0, len, kt, d, k0, k_hi);
        kv4_stage_keys<T, DH>(Vs, p.base, p.c, v_row0, len, vt, d, k0, k_hi);
        __syncthreads();
        float s[2][4];
        kv4_tile_product<DH>(Qs, Ks, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = k0 + tx + 8 * j < k_hi ? s[i][j] * p.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int x = 1; x < 8; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float mn = fmaxf(m[i], mx), mz = mn == -INFINITY ? 0.f : mn;
            const float a = exp2f(m[i] - mz);      // the tile has a key, so mn is finite unless a score is -inf
            float rs = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = exp2f(s[i][j] - mz);
                Ps[(tx + 8 * j) * 36 + 2 * ty + i] = e;
                rs += e;
            }
#pragma unroll
            for (int x = 1; x < 8; x <<= 1) rs += __shfl_xor_sync(0xffffffffu, rs, x);
            l[i] = l[i] * a + rs;
            m[i] = mn;
            if (tx == 0) al[2 * ty + i] = a;
        }
        __syncthreads();
        float av[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = al[4 * py + i];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NC; ++j) o[i][j] *= av[i];
#pragma unroll 4
        for (int k = 0; k < 32; ++k) {
            const float4 pr = *reinterpret_cast<const float4 *>(Ps + k * 36 + 4 * py);
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const float v = Vs[k * (DH + 4) + px + 16 * j];
                o[0][j] = fmaf(pr.x, v, o[0][j]);
                o[1][j] = fmaf(pr.y, v, o[1][j]);
                o[2][j] = fmaf(pr.z, v, o[2][j]);
                o[3][j] = fmaf(pr.w, v, o[3][j]);
            }
        }
    }
    __syncthreads();
    if (tx == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ls[2 * ty + i] = l[i];
            ms[2 * ty + i] = m[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * py + i, row = q0 + r;
        if (row >= p.n_q) continue;
        const float lr = ls[r], inv = lr > 0.f ? 1.f / lr : (lr == 0.f ? 0.f : lr);   // no key: 0; NaN stays
        const float lse2 = lr > 0.f ? ms[r] + log2f(lr) : (lr == 0.f ? -INFINITY : lr);
        if (p.n_split == 1) {
            T *dst = (T *)p.out + ((int64_t)b * p.n_q + row) * d + h * DH;
#pragma unroll
            for (int j = 0; j < NC; ++j) dst[px + 16 * j] = from_f<T>(o[i][j] * inv);
            if (p.lse && px == 0) p.lse[((int64_t)h * p.B + b) * p.n_q + row] = lse2 * KV4_LN2;
        } else {
            const int64_t at = (((int64_t)b * p.c.H + h) * p.n_split + sp) * p.n_q + row;
#pragma unroll
            for (int j = 0; j < NC; ++j) p.part_o[at * DH + px + 16 * j] = o[i][j] * inv;
            if (px == 0) p.part_l[at] = lse2;
        }
    }
}

// Join the partial results of the key splits: with w_s = 2^(lse_s - max),
// out = sum w_s o_s / sum w_s, lse = max + log2 sum w_s; rows without any key get
// 0 and -inf. A warp per (item, head, row), in a fixed order. grid (rows / 8, H, B).
template <typename T, int DH>
__global__ void __launch_bounds__(256) k_kv4_combine(Kv4AttnArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, row = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
    if (row >= p.n_q) return;
    const int64_t at0 = ((int64_t)b * p.c.H + h) * p.n_split * p.n_q + row;
    float m = -INFINITY;
    for (int s = lane; s < p.n_split; s += 32) m = fmaxf(m, p.part_l[at0 + (int64_t)s * p.n_q]);
    m = warp_max(m);
    const float mz = m == -INFINITY ? 0.f : m;
    float sum = 0.f, o[DH / 32];
#pragma unroll
    for (int j = 0; j < DH / 32; ++j) o[j] = 0.f;
    for (int s0 = 0; s0 < p.n_split; s0 += 32) {            // 32 weights at a time, one a lane
        const int n = min(32, p.n_split - s0);
        const float w = lane < n ? exp2f(p.part_l[at0 + (int64_t)(s0 + lane) * p.n_q] - mz) : 0.f;
        sum += warp_sum(w);
#pragma unroll 8
        for (int s = 0; s < n; ++s) {
            const float ws = __shfl_sync(0xffffffffu, w, s);
            const float *src = p.part_o + (at0 + (int64_t)(s0 + s) * p.n_q) * DH + lane;
#pragma unroll
            for (int j = 0; j < DH / 32; ++j) o[j] = fmaf(ws, src[32 * j], o[j]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int d = p.c.H * DH;
    T *dst = (T *)p.out + ((int64_t)b * p.n_q + row) * d + h * DH;
#pragma unroll
    for (int j = 0; j < DH / 32; ++j) dst[lane + 32 * j] = from_f<T>(o[j] * inv);
    if (p.lse && lane == 0)
        p.lse[((int64_t)h * p.B + b) * p.n_q + row] = sum == 0.f ? -INFINITY : (mz + log2f(sum)) * KV4_LN2;
}

// ------------------------------------------------------------------ CUDA-core scores
// out[b][h][j] = in[b][h][j] + sum_i exp(q_i . k_j / sqrt(Dh) - lse_i) for the rows
// j < len of cache item b, over the queries i of every item that reads it. 32 keys
// a CTA, every query in steps of 32; the sum over queries is the CTA's own, in a
// fixed order. grid (key tiles, H, cache items).
struct Kv4ScoreArgs {
    const uint8_t *base;
    Kv4Dims c;
    const int *prefix_len;
    int layer;
    const void *q;               // [cache items][n_q][d]
    int n_q;                     // query rows per cache item
    const float *lse;            // [H][cache items * n_q], natural log
    const float *in;             // [B][H][P] or null (zeros)
    float *out;                  // may be in
    float scale_log2;
    uint32_t *err;
    Kv4Lop lop;
};

template <int DH>
constexpr size_t kv4_scores_simt_smem() {
    return sizeof(float) * (2 * 32 * (DH + 4) + 32);
}

// The exponent's offset of a query row: log2 of its sum, +inf (weight 0) for a row
// that had no key.
__device__ __forceinline__ float kv4_lse2(float lse) {
    return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
}

template <typename T, int DH>
__global__ void __launch_bounds__(128) k_kv4_scores_simt(Kv4ScoreArgs p) {
    extern __shared__ __align__(16) float sm4[];
    float *Ks = sm4, *Qs = Ks + 32 * (DH + 4), *lq = Qs + 32 * (DH + 4);
    const int h = blockIdx.y, b = blockIdx.z, k0 = blockIdx.x * 32, d = p.c.H * DH;
    const int tid = threadIdx.x, ty = tid >> 3, tx = tid & 7;
    const int len = kv4_len(p.c, p.prefix_len, b);
    if (p.out != p.in) {
        for (int i = tid; i < 32; i += 128) {           // rows behind the item's own keep what they had
            const int j = k0 + i;
            const int64_t at = ((int64_t)b * p.c.H + h) * p.c.P + j;
            if (j >= len && j < p.c.P) p.out[at] = p.in ? p.in[at] : 0.f;
        }
    }
    if (k0 >= len) return;
    kv4_stage_keys<T, DH>(Ks, p.base, p.c, kv4_row0(p.c, p.layer, 0, b, h), len, nullptr, d, k0, len);
    const T *q = (const T *)p.q + (int64_t)b * p.n_q * d + h * DH;
    const float *lse = p.lse + ((int64_t)h * p.c.B + b) * p.n_q;
    float sum[2] = {0.f, 0.f};
    for (int q0 = 0; q0 < p.n_q; q0 += 32) {
        __syncthreads();
        kv4_stage_rows<T, DH>(Qs, q, q0, p.n_q, d);
        if (tid < 32) lq[tid] = q0 + tid < p.n_q ? kv4_lse2(lse[q0 + tid]) : INFINITY;
        __syncthreads();
        float s[2][4];
        kv4_tile_product<DH>(Ks, Qs, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[i] += exp2f(s[i][j] * p.scale_log2 - lq[tx + 8 * j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float t = sum[i];
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
        const int j = k0 + 2 * ty + i;
        if (tx == 0 && j < len) {
            const int64_t at = ((int64_t)b * p.c.H + h) * p.c.P + j;
            p.out[at] = (p.in ? p.in[at] : 0.f) + t;
        }
    }
}

}  // namespace qi21
