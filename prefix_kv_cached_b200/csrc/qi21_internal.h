// Internal declarations shared by the host helpers and the CUDA entry points.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "qi21.h"

namespace qi21 {

// Workspace carve-up. Every region starts on a 256-byte boundary.
//   err     : device error words (uint32 [8])
//   gates   : fp32 [4][d]  tanh(gate1) prefix row, tanh(gate1) target row,
//                          tanh(gate2) prefix row, tanh(gate2) target row
//   modtmp  : fp32 [2][d]  timestep-MLP intermediates
//   h       : fp32 [R][d]  residual stream (R = B * S rows at most)
//   xn      : T [R][d]     modulated LayerNorm output (LN1 and LN2 share it)
//   q       : T [R][d]     queries after QK-RMSNorm and RoPE
//   o       : T [R][d]     attention output
//   hid     : T [R][F]     SwiGLU activation
//   kvf     : T [2][B][S][d]  K/V of the full recomputation
//   gemm    : fp32 [R][max(3d, 2F)]  outputs of the CUDA-core GEMMs (present when
//             they run: F32 mode, or BF16 mode with the tensor cores switched off)
//   xin     : bf16 [B*N][C]   the latent rounded for the tensor-core img_in
//   fwp, fu : bf16 [C][d], fp32 [C]  W_out scaled by (1 + scale_final) and its row
//             sums (tensor-core final AdaLN + proj_out)
//   fpart   : fp32 [FINAL_MAX_KSPLIT][B*N][68]  its per-K-slice partial sums
constexpr int FINAL_MAX_KSPLIT = 8;
struct WsLayout {
    size_t err, gates, modtmp, h, xn, q, o, hid, kvf, gemm, xin, fwp, fu, fpart, total;
};

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

inline size_t dtype_bytes(int32_t dtype) { return dtype == QI21_DTYPE_BF16 ? 2 : 4; }

// Kernel family of the BF16 mode (process-wide; qi21_set_tensor_cores).
bool tc_enabled();

// The shape checks every device entry point applies before enqueueing work:
// QI21_ERR_INVALID_ARG / SHAPE / UNSUPPORTED, or QI21_OK.
qi21_status check_config_shapes(const qi21_config *c);

// Packed weight buffer of qi21_pack_weights: the 15 tensors of qi21_weights in
// struct order, [out][in] (stacked [L][out][in]), each on a 256-byte boundary.
struct PackedLayout {
    size_t off[15];
    size_t total;
};
inline PackedLayout packed_layout(const qi21_config &c) {
    const size_t eb = dtype_bytes(c.dtype);
    const size_t d = c.d_model, C = c.latent_ch, T = c.time_dim, F = c.mlp_hidden, L = c.n_layers;
    const size_t nch = c.use_shift ? 6 : 4, dh = c.head_dim;
    const size_t sizes[15] = {d * C * eb,     C * d * eb,     d * T * eb,     d * d * eb,     nch * d * d * eb,
                              d * d * eb,     L * d * d * eb, L * d * d * eb, L * d * d * eb, L * d * d * eb,
                              L * F * d * eb, L * F * d * eb, L * d * F * eb, L * dh * 4,     L * dh * 4};
    PackedLayout p{};
    size_t o = 0;
    for (int i = 0; i < 15; ++i) {
        p.off[i] = o;
        o += align256(sizes[i]);
    }
    p.total = o;
    return p;
}

inline bool uses_cuda_core_gemm(const qi21_config &c) { return c.dtype == QI21_DTYPE_F32 || !tc_enabled(); }

inline WsLayout ws_layout(const qi21_config &c, int64_t B, int64_t P, int64_t N) {
    const int64_t S = P + N, R = B * S, d = c.d_model, F = c.mlp_hidden;
    const size_t eb = dtype_bytes(c.dtype);
    WsLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        size_t o = off;
        off += align256(bytes);
        return o;
    };
    L.err = take(64);
    L.gates = take(sizeof(float) * 4 * d);
    L.modtmp = take(sizeof(float) * 2 * d);
    L.h = take(sizeof(float) * R * d);
    L.xn = take(eb * R * d);
    L.q = take(eb * R * d);
    L.o = take(eb * R * d);
    L.hid = take(eb * R * F);
    L.kvf = take(eb * 2 * B * S * d);
    const int64_t gw = (3 * d > 2 * F) ? 3 * d : 2 * F;
    L.gemm = take(uses_cuda_core_gemm(c) ? sizeof(float) * R * gw : 0);
    const int64_t C = c.latent_ch;
    L.xin = take(2 * B * N * C);
    L.fwp = take(2 * C * d);
    L.fu = take(sizeof(float) * C);
    L.fpart = take(sizeof(float) * FINAL_MAX_KSPLIT * B * N * 68);
    L.total = off;
    return L;
}

// Plan of an attention over a 4-bit cache: which kernel, how the work is cut, and
// the fp32 partial results (log2-sum-exp, then normalised outputs) in the
// workspace. Host arithmetic on sizes alone, so that the size query and the call
// agree (items: those of the cache, B or 1); 148 is the number of SMs the cuts are made for, not one they need.
//   Kv4Work: the tensor-core kernel's steps. A step is one 128-key tile of one unit
//   (item, head, unit_rows query rows); `units` units of `tiles` steps each, laid
//   end to end, are shared out over `grid` CTAs: evenly, or (whole = 1) in whole
//   units. slot_rows: rows of a partial-result slot, two slots a CTA.
struct Kv4Work {
    int units, tiles_p, tiles, grid, whole;
    int q_tiles, unit_rows, slot_rows;
};

//   expanded: the layer's prefix rows are first written out in bf16 (expand, [K|V]
//   [items][Pp][d]) and the attention reads those.
//   rows: few query rows; CTAs of 8 or 16 rows whose keys are split.
struct Kv4Plan {
    bool tc, expanded, rows, cluster, ok;
    int n_split;                 // rows and CUDA-core kernels: parts the keys are split into
    Kv4Work w;
    size_t part_l, part_o, expand, total;
};

constexpr int KV4_SMS = 148;
// A cut costs a pass over the partial results (about 4 us, as long as four steps of
// 1 us each); whole units are taken where the even share is not that much shorter.
constexpr int KV4_CUT_STEPS = 4;

// The prefix is expanded once, instead of for every 256 rows, from KV4_EXPAND_ROWS
// query rows on, where the 128-row query tiles fill the SMs, the prefix is no less than
// the tail, and its bf16 copy stays in L2; where it does not, above twice the rows, since
// up to there the copy's memory buys nothing. us, expanded / not, 32 heads of 128, as
// many tail keys as rows: P 4608: 4096 rows 459 / 530, 2048 rows 200 / 232, 1024 rows 97
// / 120, 512 rows 69 / 69; P 33792 (a copy of 553 MB): 1024 rows 628 / 559, 2048 rows
// 1069 / 1070, 2176 rows 1093 / 1170, 2432 rows 1486 / 1469, 2944 rows 1497 / 1855, 4096
// rows 2145 / 2490; P 12000 (197 MB): 2048 rows 508 / 523, 2304 rows 517 / 572. 8 x 16
// heads of 64, P 512: 2048 rows 310 / 286; P 8000 (262 MB): 2304 rows 1190 / 1247.
constexpr int KV4_EXPAND_ROWS = 1024;
constexpr int64_t KV4_EXPAND_L2 = 96 << 20;     // of 126 MB
// Up to this many query rows the few-rows kernels. us, 32 heads of 128, P 33792:
// attention 16 rows 62, 32 rows 111, the tensor-core kernel 105 at 32 and 64 rows (but
// 15 against 8 at 32 rows over 1032 keys of 16 heads of 64); weights 16 rows 46, 32 rows 76, the tensor-core kernel 129 at 33.
constexpr int KV4_ROWS_MAX = 32;
// Key splits that a cluster merges: the portable cluster size.
constexpr int KV4_ROWS_CLUSTER = 8;

inline Kv4Plan kv4_plan(const qi21_config &c, int64_t items, int64_t B, int64_t n_q, int64_t P, int64_t n_tail) {
    Kv4Plan p{};
    const int64_t keys = P + n_tail, H = c.n_heads;
    size_t rows = 0;             // rows of partial results
    p.ok = true;
    p.tc = c.dtype == QI21_DTYPE_BF16 && tc_enabled();
    if (p.tc && n_q <= KV4_ROWS_MAX) {
        // three CTAs of 8 rows or two of 16 an SM, at least a 64-key chunk for each of a
        // CTA's four warps
        p.rows = true;
        const int64_t tile = n_q <= 8 ? 8 : 16, ctas = (n_q + tile - 1) / tile * H * B;
        const int64_t chunks = (P + 63) / 64 + (n_tail + 63) / 64;
        int64_t n = (tile == 8 ? 3 : 2) * KV4_SMS / ctas;
        if (n > (chunks + 3) / 4) n = (chunks + 3) / 4;
        // merged within a cluster, without a second pass over partial results, where that
        // costs at most an eighth of the splits (one row, 32 heads of 128, P 33792: 13
        // splits and the pass 55 us, 8 in a cluster 66; 16 rows: 9 and the pass 66, 8 62)
        p.cluster = n > 1 && n <= KV4_ROWS_CLUSTER + KV4_ROWS_CLUSTER / 8;
        if (p.cluster && n > KV4_ROWS_CLUSTER) n = KV4_ROWS_CLUSTER;
        p.n_split = (int)(n < 1 ? 1 : n);
        if (B * p.n_split > 65535) p.ok = false;
        rows = p.n_split > 1 && !p.cluster ? (size_t)(B * H * n_q) * p.n_split : 0;
    } else if (p.tc) {
        const int64_t ur = n_q <= 128 ? 128 : 256, qt = (n_q + ur - 1) / ur, units = B * H * qt;
        const int64_t tp = (P + 127) / 128, tiles = tp + (n_tail + 127) / 128, steps = units * tiles;
        const int64_t grid = steps < KV4_SMS ? steps : KV4_SMS;
        const int64_t grid_w = units < KV4_SMS ? units : KV4_SMS;
        p.w.whole = (units + grid_w - 1) / grid_w * tiles <= (steps + grid - 1) / grid + KV4_CUT_STEPS;
        p.w.units = (int)units;
        p.w.tiles_p = (int)tp;
        p.w.tiles = (int)tiles;
        p.w.grid = (int)(p.w.whole ? grid_w : grid);
        p.w.q_tiles = (int)qt;
        p.w.unit_rows = (int)ur;
        p.w.slot_rows = (int)(qt == 1 ? n_q : ur);
        if (units > INT32_MAX) p.ok = false;
        const int64_t copy = 4 * items * tp * 128 * c.d_model;
        p.expanded = (copy <= KV4_EXPAND_L2 ? n_q >= KV4_EXPAND_ROWS : n_q > 2 * KV4_EXPAND_ROWS) && P >= n_tail &&
                     B * H * ((n_q + 127) / 128) >= KV4_SMS;
        if (p.expanded && (B > 65535 || (n_q + 127) / 128 > INT32_MAX)) p.ok = false;
        rows = p.w.whole || p.expanded ? 0 : (size_t)2 * p.w.grid * p.w.slot_rows;
    } else {
        // CTAs of 32 query rows; two CTAs an SM, at least 64 keys each
        const int64_t ctas = (n_q + 31) / 32 * H * B;
        int64_t n = (2 * KV4_SMS + ctas - 1) / ctas;
        if (n > (keys + 63) / 64) n = (keys + 63) / 64;
        p.n_split = (int)(n < 1 ? 1 : n);
        if (B * p.n_split > 65535) p.ok = false;
        rows = p.n_split > 1 ? (size_t)(B * H * n_q) * p.n_split : 0;
    }
    p.part_l = 256;
    p.part_o = p.part_l + align256(rows * 4);
    p.expand = p.part_o + align256(rows * 4 * c.head_dim);
    p.total = p.expand;
    if (p.expanded) p.total += align256((size_t)2 * items * ((P + 127) / 128 * 128) * c.d_model * 2);
    return p;
}

// Plan of the accumulated weights: the tensor-core kernel's CTAs take one 128-key
// tile each; where those are fewer than two an SM, the query tiles are split, whose
// sums lie in the workspace.
//   rows: few query rows; n_split is then the parts a head's keys are split into, and
//   no sum is split.
struct Kv4ScorePlan {
    bool tc, rows, ok;
    int q_tiles, n_split;
    size_t part, total;
};

// rows: query rows per cache item
inline Kv4ScorePlan kv4_score_plan(const qi21_config &c, int64_t items, int64_t rows, int64_t P) {
    Kv4ScorePlan p{};
    p.tc = c.dtype == QI21_DTYPE_BF16 && tc_enabled();
    p.n_split = 1;
    p.ok = items <= 65535;
    p.part = p.total = 256;
    if (p.tc && rows <= KV4_ROWS_MAX) {
        p.rows = true;
        int64_t n = 4 * KV4_SMS / (c.n_heads * items);         // four CTAs an SM
        const int64_t most = (P + 255) / 256;                  // a 64-key chunk for each warp
        if (n > most) n = most;
        p.n_split = (int)(n < 1 ? 1 : n);
    } else if (p.tc) {
        const int64_t tp = (P + 127) / 128, ctas = tp * c.n_heads * items, qt = (rows + 127) / 128;
        int64_t n = (2 * KV4_SMS) / ctas;
        if (n > qt) n = qt;
        p.n_split = (int)(n < 1 ? 1 : n);
        p.q_tiles = (int)qt;
        if (items * p.n_split > 65535) p.ok = false;
        if (p.n_split > 1) p.total += align256((size_t)p.n_split * items * c.n_heads * tp * 128 * 4);
    }
    return p;
}

// Workspace of the attention and of the weights, over a cache of B items or of one
// that B requests share.
inline size_t kv4_ops_workspace(const qi21_config &c, int64_t B, int64_t n_q, int64_t P, int64_t n_tail) {
    size_t most = 0;
    for (int64_t items = 1; items <= B; items += B > 1 ? B - 1 : 1) {
        const size_t a = kv4_plan(c, items, B, n_q, P, n_tail).total;
        const size_t s = kv4_score_plan(c, items, items == 1 ? B * n_q : n_q, P).total;
        most = most > a ? most : a;
        most = most > s ? most : s;
    }
    return most;
}

// Workspace of the cached step over a 4-bit cache: that of a cached step without
// prefix (its full-recompute K/V region holds the target K/V), the rows'
// log-sum-exps, and the attention's partial results.
struct Kv4StepLayout {
    size_t lse, kv4, total;
};

inline Kv4StepLayout kv4_step_layout(const qi21_config &c, int64_t B, int64_t P, int64_t N) {
    Kv4StepLayout s{};
    s.lse = ws_layout(c, B, 0, N).total;
    s.kv4 = s.lse + align256(sizeof(float) * (size_t)c.n_heads * B * N);
    s.total = s.kv4 + kv4_ops_workspace(c, B, N, P, N);
    return s;
}

inline bool kv4_head_dim_ok(const qi21_config &c) {
    return c.head_dim % QI21_KV4_GROUP == 0 && c.head_dim <= 128;
}

}  // namespace qi21
