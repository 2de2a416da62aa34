// Launches of the 4-bit prefix cache's operators and their argument checks
// (included by qi21_api.cu; the kernels are in qi21_kv4.cuh, qi21_kv4_attn_tc.cuh,
// qi21_kv4_rows.cuh, qi21_kv4_scores_tc.cuh and, over the expanded prefix,
// qi21_attn_tc.cuh).
#pragma once
#include "qi21_kv4.cuh"
#include "qi21_kv4_attn_tc.cuh"
#include "qi21_kv4_rows.cuh"
#include "qi21_kv4_scores_tc.cuh"

namespace qi21 {

static Kv4Dims kv4_dims(const qi21_kv4_cache &k) {
    Kv4Dims c{};
    c.B = k.batch;
    c.H = k.n_heads;
    c.P = k.n_prefix;
    c.Pp = (int)kv4_pad(k.n_prefix);
    c.Dh = k.head_dim;
    c.scales_off = (int64_t)k.n_layers * 2 * c.B * c.H * c.Pp * (c.Dh / 2);
    return c;
}

// A cache descriptor against the config: sizes that match and fit the launches.
static qi21_status check_kv4(const qi21_config *c, const qi21_kv4_cache *k) {
    if (!k || !al16(k->base) || ((uintptr_t)k->prefix_len & 15)) return QI21_ERR_INVALID_ARG;
    if (!kv4_head_dim_ok(*c)) return QI21_ERR_UNSUPPORTED;
    if (k->n_layers != c->n_layers || k->n_heads != c->n_heads || k->head_dim != c->head_dim || k->batch <= 0 ||
        k->n_prefix <= 0 || k->n_prefix > INT32_MAX - 128)
        return QI21_ERR_CACHE_STATE;
    if ((int64_t)k->n_layers * 2 * k->batch > 65535 || k->n_heads > 65535) return QI21_ERR_SHAPE;
    // a slab's units of 32 elements are counted in 32 bits
    if (((int64_t)k->n_prefix + 131) / 4 * (c->d_model / 8) > UINT32_MAX - 256ll) return QI21_ERR_SHAPE;
    return QI21_OK;
}

// A token-major cache and a 4-bit one that hold the same prefix rows.
static bool kv4_matches(const qi21_config *c, const qi21_kv_cache *a, const qi21_kv4_cache *k) {
    return a->n_layers == c->n_layers && a->d_model == c->d_model && a->dtype == c->dtype && a->batch > 0 &&
           a->n_target > 0 && a->n_prefix == k->n_prefix && k->batch == (a->shared_prefix ? 1 : a->batch);
}

static int64_t kv_slab_rows(const qi21_kv_cache &a) {
    return a.shared_prefix ? kv4_pad(a.n_prefix) + (int64_t)a.batch * a.n_target
                           : (int64_t)a.n_prefix + a.n_target;
}

// A thread for every `rows` rows by `dims` dims of a slab.
static dim3 kv4_row_grid(const qi21_config &c, const qi21_kv4_cache &k, int rows, int dims) {
    const int64_t units = ((int64_t)k.n_prefix + rows - 1) / rows * (c.d_model / dims);
    return dim3((unsigned)((units + 255) / 256), (unsigned)(c.n_layers * 2 * k.batch));
}

template <typename T>
static void launch_kv4_quantize(Launcher &L, const qi21_config &c, const qi21_kv_cache &src,
                                const qi21_kv4_cache &dst) {
    L.run("kv4_quantize", [&] {
        launch_dep(k_kv4_quantize<T>, kv4_row_grid(c, dst, KV4_Q_ROWS, 16), dim3(256), 0, L.st, nullptr, (const T *)src.base,
                   kv_slab_rows(src) * c.d_model, kv4_dims(dst), dst.prefix_len, (uint8_t *)dst.base);
    });
}

template <typename T>
static void launch_kv4_dequantize(Launcher &L, const qi21_config &c, const qi21_kv4_cache &src,
                                  const qi21_kv_cache &dst) {
    L.run("kv4_dequantize", [&] {
        launch_dep(k_kv4_dequantize<T>, kv4_row_grid(c, src, KV4_D_ROWS, 8), dim3(256), 0, L.st, nullptr, (const uint8_t *)src.base,
                   kv4_dims(src), 0, src.prefix_len, 0, (T *)dst.base, kv_slab_rows(dst) * c.d_model, kKv4Lop);
    });
}

template <typename T, int DH>
static void launch_kv4_attn_simt(Launcher &L, const Kv4AttnArgs &p) {
    constexpr size_t smem = kv4_attn_simt_smem<DH>();
    static DeviceFlags attr;
    smem_opt_in(k_kv4_attn_simt<T, DH>, (int)smem, attr);
    L.run("kv4_attn_simt", [&] {
        k_kv4_attn_simt<T, DH><<<dim3((p.n_q + 31) / 32, p.c.H, p.B * p.n_split), 128, smem, L.st>>>(p);
    });
    if (p.n_split > 1)
        L.run("kv4_combine", [&] {
            k_kv4_combine<T, DH><<<dim3((p.n_q + 7) / 8, p.c.H, p.B), 256, 0, L.st>>>(p);
        });
}

template <int DH>
static void launch_kv4_attn_tc(Launcher &L, const Kv4AttnArgs &a, const Kv4Plan &plan) {
    const uint64_t d = (uint64_t)a.c.H * DH, n_q = a.n_q, nt = a.n_tail > 0 ? a.n_tail : n_q;
    CUtensorMap q, k, v;
    // without a tail its maps are never used; they only have to be valid
    if (!make_map4(&q, a.q, d, n_q, a.B, 1, d, n_q * d, a.B * n_q * d) ||
        !make_map4(&k, a.n_tail > 0 ? a.k_tail : a.q, d, nt, a.B, 1, d, nt * d, a.B * nt * d) ||
        !make_map4(&v, a.n_tail > 0 ? a.v_tail : a.q, d, nt, a.B, 1, d, nt * d, a.B * nt * d)) {
        L.status = QI21_ERR_CUDA;
        return;
    }
    Kv4TcArgs p{};
    p.a = a;
    p.w = plan.w;
    p.part_l = a.part_l;
    p.part_o = a.part_o;
    using C = Kv4AttnCfg<DH>;
    auto go = [&](auto *kernel, DeviceFlags &attr) {
        smem_opt_in(kernel, (int)C::SMEM, attr);
        L.run("kv4_attn", [&] {
            launch_dep(kernel, dim3(p.w.grid), dim3(C::THREADS), C::SMEM, L.st, nullptr, q, k, v, p);
        });
    };
    if (p.w.unit_rows == 128) {
        static DeviceFlags attr;
        go(k_kv4_attn_tc<DH, true>, attr);
    } else {
        static DeviceFlags attr;
        go(k_kv4_attn_tc<DH, false>, attr);
    }
    if (!p.w.whole && p.w.grid > 1)
        L.run("kv4_join", [&] {
            launch_dep(k_kv4_join<DH>, dim3((p.w.slot_rows + 8 * KV4_JOIN_ROWS - 1) / (8 * KV4_JOIN_ROWS), p.w.grid - 1),
                       dim3(256), 0, L.st, nullptr, p);
        });
}

template <int DH>
static void launch_kv4_attn_rows(Launcher &L, const Kv4AttnArgs &p) {
    constexpr size_t smem = Kv4RowsCfg<DH, true>::SMEM;
    auto go = [&](auto *kernel, int tile, DeviceFlags &attr) {
        smem_opt_in(kernel, (int)smem, attr);
        cudaLaunchAttribute cl;
        cl.id = cudaLaunchAttributeClusterDimension;
        cl.val.clusterDim.x = 1;
        cl.val.clusterDim.y = 1;
        cl.val.clusterDim.z = p.n_split;
        L.run("kv4_attn", [&] {
            launch_dep(kernel, dim3((p.n_q + tile - 1) / tile, p.c.H, p.B * p.n_split), dim3(32 * KV4R_WARPS), smem, L.st,
                       p.cluster ? &cl : nullptr, p);
        });
    };
    if (p.n_q <= 8) {
        static DeviceFlags attr;
        go(k_kv4_attn_rows<DH, 1>, 8, attr);
    } else {
        static DeviceFlags attr;
        go(k_kv4_attn_rows<DH, 2>, 16, attr);
    }
    if (p.n_split > 1 && !p.cluster)
        L.run("kv4_combine", [&] {
            launch_dep(k_kv4_combine<bf16, DH>, dim3((p.n_q + 7) / 8, p.c.H, p.B), dim3(256), 0, L.st, nullptr, p);
        });
}

// Many query rows: the layer's prefix in bf16 first, then the attention over it
// and the tail.
template <int DH>
static void launch_kv4_attn_expanded(Launcher &L, const Kv4AttnArgs &a, const Kv4Plan &plan, char *ws) {
    const uint64_t d = (uint64_t)a.c.H * DH, n_q = a.n_q, nt = a.n_tail > 0 ? a.n_tail : n_q, pp = a.c.Pp;
    bf16 *ek = (bf16 *)(ws + plan.expand), *ev = ek + a.c.B * pp * d;
    const int64_t quads = pp / KV4_D_ROWS;
    L.run("kv4_expand", [&] {
        launch_dep(k_kv4_dequantize<bf16>, dim3((unsigned)((quads * (d / 8) + 255) / 256), 2 * a.c.B), dim3(256), 0,
                   L.st, nullptr, a.base, a.c, a.layer * 2 * a.c.B, a.prefix_len, 1, ek, (int64_t)(pp * d), kKv4Lop);
    });
    CUtensorMap q, k, v, kt, vt;
    if (!make_map4(&q, a.q, d, n_q, a.B, 1, d, n_q * d, a.B * n_q * d) ||
        !make_map4(&k, ek, d, pp, a.c.B, 1, d, pp * d, a.c.B * pp * d) ||
        !make_map4(&v, ev, d, pp, a.c.B, 1, d, pp * d, a.c.B * pp * d) ||
        // without a tail its maps are never used; they only have to be valid
        !make_map4(&kt, a.n_tail > 0 ? a.k_tail : a.q, d, nt, a.B, 1, d, nt * d, a.B * nt * d) ||
        !make_map4(&vt, a.n_tail > 0 ? a.v_tail : a.q, d, nt, a.B, 1, d, nt * d, a.B * nt * d)) {
        L.status = QI21_ERR_CUDA;
        return;
    }
    AttnParams p{};
    p.Mq = a.n_q;
    p.kv_len = a.c.P + a.n_tail;
    p.H = a.c.H;
    p.d = (int)d;
    p.out = (bf16 *)a.out;
    p.scale_log2 = a.scale_log2;
    p.err = a.err;
    p.prefix_len = a.c.P;
    p.tgt_len = a.n_tail;
    const AttnExt x{a.prefix_len, a.shared, a.lse};
    using Cf = AttnCfg<DH>;
    static DeviceFlags attr;
    smem_opt_in(k_attn_tc_ext<DH>, (int)Cf::SMEM, attr);
    L.run("kv4_attn", [&] {
        launch_dep(k_attn_tc_ext<DH>, dim3((p.Mq + Cf::BQ - 1) / Cf::BQ, p.H, a.B), dim3(Cf::THREADS), Cf::SMEM, L.st,
                   nullptr, q, k, v, kt, vt, p, x);
    });
}

// Attention of one layer; ws: the region that kv4_plan() lays out.
template <typename T>
static void launch_kv4_attention(Launcher &L, const qi21_config &c, const qi21_kv4_cache &k, int layer, const void *q,
                                 int B, int n_q, const void *k_tail, const void *v_tail, int n_tail, void *out,
                                 float *lse, char *ws, uint32_t *err) {
    const Kv4Plan plan = kv4_plan(c, k.batch, B, n_q, k.n_prefix, n_tail);
    Kv4AttnArgs p{};
    p.base = (const uint8_t *)k.base;
    p.c = kv4_dims(k);
    p.prefix_len = k.prefix_len;
    p.layer = layer;
    p.shared = k.batch == 1;
    p.q = q;
    p.B = B;
    p.n_q = n_q;
    p.k_tail = k_tail;
    p.v_tail = v_tail;
    p.n_tail = n_tail;
    p.out = out;
    p.lse = lse;
    p.n_split = plan.n_split;
    p.cluster = plan.cluster;
    p.part_l = (float *)(ws + plan.part_l);
    p.part_o = (float *)(ws + plan.part_o);
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)c.head_dim);
    p.err = err;
    p.lop = kKv4Lop;
    if (plan.rows) {
        if (c.head_dim == 64)
            launch_kv4_attn_rows<64>(L, p);
        else
            launch_kv4_attn_rows<128>(L, p);
        return;
    }
    if (plan.expanded) {
        if (c.head_dim == 64)
            launch_kv4_attn_expanded<64>(L, p, plan, ws);
        else
            launch_kv4_attn_expanded<128>(L, p, plan, ws);
        return;
    }
    if (plan.tc) {
        if (c.head_dim == 64)
            launch_kv4_attn_tc<64>(L, p, plan);
        else
            launch_kv4_attn_tc<128>(L, p, plan);
        return;
    }
    switch (c.head_dim) {
        case 32: launch_kv4_attn_simt<T, 32>(L, p); break;
        case 64: launch_kv4_attn_simt<T, 64>(L, p); break;
        case 96: launch_kv4_attn_simt<T, 96>(L, p); break;
        default: launch_kv4_attn_simt<T, 128>(L, p); break;
    }
}

template <typename T, int DH>
static void launch_kv4_scores_simt(Launcher &L, const Kv4ScoreArgs &p) {
    constexpr size_t smem = kv4_scores_simt_smem<DH>();
    static DeviceFlags attr;
    smem_opt_in(k_kv4_scores_simt<T, DH>, (int)smem, attr);
    L.run("kv4_scores_simt", [&] {
        k_kv4_scores_simt<T, DH><<<dim3((p.c.P + 31) / 32, p.c.H, p.c.B), 128, smem, L.st>>>(p);
    });
}

template <int DH>
static void launch_kv4_scores_tc(Launcher &L, const Kv4ScoreArgs &a, const Kv4ScorePlan &plan, float *part) {
    const uint64_t d = (uint64_t)a.c.H * DH, n_q = a.n_q;
    CUtensorMap q;
    if (!make_map4(&q, a.q, d, n_q, a.c.B, 1, d, n_q * d, a.c.B * n_q * d)) {
        L.status = QI21_ERR_CUDA;
        return;
    }
    Kv4ScoreTcArgs p{a, plan.q_tiles, plan.n_split, part};
    using C = Kv4ScoreCfg<DH>;
    static DeviceFlags attr;
    smem_opt_in(k_kv4_scores_tc<DH>, (int)C::SMEM, attr);
    L.run("kv4_scores", [&] {
        launch_dep(k_kv4_scores_tc<DH>, dim3(a.c.Pp / 128, a.c.H, a.c.B * p.n_split), dim3(C::THREADS), C::SMEM, L.st,
                   nullptr, q, p);
    });
    if (p.n_split > 1)
        L.run("kv4_scores_reduce", [&] {
            launch_dep(k_kv4_scores_reduce, dim3((a.c.P + 255) / 256, a.c.H, a.c.B), dim3(256), 0, L.st, nullptr, p);
        });
}

template <int DH>
static void launch_kv4_scores_rows(Launcher &L, const Kv4ScoreArgs &p, int n_split) {
    constexpr size_t smem = Kv4RowsCfg<DH, false>::SMEM;
    static DeviceFlags attr;
    smem_opt_in(k_kv4_scores_rows<DH>, (int)smem, attr);
    L.run("kv4_scores", [&] {
        launch_dep(k_kv4_scores_rows<DH>, dim3(n_split, p.c.H, p.c.B), dim3(32 * KV4R_WARPS), smem, L.st, nullptr, p);
    });
}

template <typename T>
static void launch_kv4_scores(Launcher &L, const qi21_config &c, const qi21_kv4_cache &k, int layer, const void *q,
                              int B, int n_q, const float *lse, const float *in, float *out, char *ws,
                              uint32_t *err) {
    Kv4ScoreArgs p{};
    p.base = (const uint8_t *)k.base;
    p.c = kv4_dims(k);
    p.prefix_len = k.prefix_len;
    p.layer = layer;
    p.q = q;
    p.n_q = k.batch == 1 ? B * n_q : n_q;      // one item: the rows of every request that reads it
    p.lse = lse;
    p.in = in;
    p.out = out;
    p.scale_log2 = 1.4426950408889634f / sqrtf((float)c.head_dim);
    p.err = err;
    p.lop = kKv4Lop;
    const Kv4ScorePlan plan = kv4_score_plan(c, k.batch, p.n_q, k.n_prefix);
    if (plan.rows) {
        if (c.head_dim == 64)
            launch_kv4_scores_rows<64>(L, p, plan.n_split);
        else
            launch_kv4_scores_rows<128>(L, p, plan.n_split);
        return;
    }
    if (plan.tc) {
        if (c.head_dim == 64)
            launch_kv4_scores_tc<64>(L, p, plan, (float *)(ws + plan.part));
        else
            launch_kv4_scores_tc<128>(L, p, plan, (float *)(ws + plan.part));
        return;
    }
    switch (c.head_dim) {
        case 32: launch_kv4_scores_simt<T, 32>(L, p); break;
        case 64: launch_kv4_scores_simt<T, 64>(L, p); break;
        case 96: launch_kv4_scores_simt<T, 96>(L, p); break;
        default: launch_kv4_scores_simt<T, 128>(L, p); break;
    }
}

constexpr int KV4_EVICT_HEADS = KV4_SMS;

static void launch_kv4_evict(Launcher &L, const qi21_config &c, const qi21_kv4_cache &src, const float *scores,
                             int keep, int n_protected, const qi21_kv4_cache &dst, int *kept) {
    const Kv4Dims cd = kv4_dims(src), od = kv4_dims(dst);
    // From a head an SM on, a block copies the rows of the head it has selected; fewer
    // heads leave SMs without a copy to make, and the rows are copied by a grid of their
    // own. us, one kernel / two: 1024 heads 512 -> 333 rows 16.5 / 19.7, 256 heads 4608 ->
    // 2304 rows 50.7 / 51.7, 1024 heads 155.7 / 166.3; 64 heads 27.8 / 27.0.
    const bool one = (int64_t)c.n_layers * cd.B * cd.H >= KV4_EVICT_HEADS;
    L.run(one ? "kv4_evict" : "kv4_select", [&] {
        // rows a thread holds: as many as the prefix needs, so that it is read once
        auto go = [&](auto *kernel, int threads) {
            launch_dep(kernel, dim3(cd.H, cd.B, c.n_layers), dim3(threads), 0, L.st, nullptr, scores, cd,
                       src.prefix_len, keep, n_protected, kept, dst.prefix_len, (const uint8_t *)src.base,
                       (uint8_t *)dst.base, od);
        };
        if (cd.P <= 512) one ? go(k_kv4_select<128, 4, true>, 128) : go(k_kv4_select<128, 4, false>, 128);
        else if (cd.P <= 2048) one ? go(k_kv4_select<256, 8, true>, 256) : go(k_kv4_select<256, 8, false>, 256);
        else one ? go(k_kv4_select<512, 16, true>, 512) : go(k_kv4_select<512, 16, false>, 512);
    });
    if (one) return;
    L.run("kv4_gather", [&] {
        const int rows = KV4_GATHER * (256 / (cd.Dh / KV4_GROUP));           // of a block
        launch_dep(k_kv4_gather, dim3((keep + rows - 1) / rows, cd.H, c.n_layers * cd.B), dim3(256), 0, L.st, nullptr,
                   (const uint8_t *)src.base, cd, kept, keep, (uint8_t *)dst.base, od);
    });
}

// Shared checks of the attention, the scores and the cached step.
static qi21_status check_kv4_queries(const qi21_config *c, const qi21_kv4_cache *k, int32_t B, int32_t n_q,
                                     int32_t n_tail) {
    qi21_status s = check_kv4(c, k);
    if (s) return s;
    if (k->state != QI21_CACHE_EXTRACTED) return QI21_ERR_CACHE_STATE;
    if (B <= 0 || n_q <= 0 || n_tail < 0) return QI21_ERR_SHAPE;
    if (k->batch != B && k->batch != 1) return QI21_ERR_CACHE_STATE;
    // one 32-bit index holds every query row, and every key of an item
    if ((int64_t)B * n_q > INT32_MAX - 256 || (int64_t)k->n_prefix + n_tail > INT32_MAX - 256) return QI21_ERR_SHAPE;
    if (!kv4_plan(*c, k->batch, B, n_q, k->n_prefix, n_tail).ok) return QI21_ERR_SHAPE;
    return QI21_OK;
}

}  // namespace qi21
