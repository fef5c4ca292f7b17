// api_block.hip -- the C ABI of what stands around the layer: products with an
// epilogue, block norms, clipping.  Validation is pure host code and comes before
// any HIP call; nothing allocates, waits or throws.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "kernels_block.h"
#include "moe_lora.h"

using namespace moe_lora;

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check(hipError_t e) { return e == hipSuccess ? MOE_LORA_OK : MOE_LORA_ERR_HIP; }

#define MOE_TRY(expr)           \
    do {                        \
        const int rc_ = (expr); \
        if (rc_ != MOE_LORA_OK) \
            return rc_;         \
    } while (0)

int check_workspace(const void *workspace, size_t bytes, size_t need)
{
    if (need == 0)
        return MOE_LORA_OK;
    if (!workspace)
        return MOE_LORA_ERR_INVALID_ARG;
    if (bytes < need)
        return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
    return aligned(workspace, kAlign) ? MOE_LORA_OK : MOE_LORA_ERR_MISALIGNED;
}

// ---- products -------------------------------------------------------------

int validate(const moe_lora_linear_shape *s)
{
    if (!s)
        return MOE_LORA_ERR_INVALID_ARG;
    if (s->rows < 0 || s->rows > 1 << 24 || s->in_features < 8 || s->in_features > 131072 ||
        s->in_features % 8 != 0 || s->out_features < 1 || s->out_features > 131072)
        return MOE_LORA_ERR_UNSUPPORTED_SHAPE;
    // launches count tiles and threads in 32 bits
    const int64_t widest = std::max<int64_t>(s->in_features, 2 * (int64_t)s->out_features);
    if (s->rows * widest > (int64_t)1 << 37)
        return MOE_LORA_ERR_UNSUPPORTED_SHAPE;
    if (s->activation < MOE_LORA_ACT_NONE || s->activation > MOE_LORA_ACT_SWIGLU ||
        (s->out_fp32 != 0 && s->out_fp32 != 1))
        return MOE_LORA_ERR_INVALID_ARG;
    return MOE_LORA_OK;
}

// A linear layer's sizes as the products see them
struct Sizes {
    int64_t M, K;
    int N, half, sets;
    bool gated;
    explicit Sizes(const moe_lora_linear_shape *s)
        : M(s->rows), K(s->in_features), N(s->out_features), half((N + 7) / 8 * 8),
          sets(s->activation == MOE_LORA_ACT_SWIGLU ? 2 : 1), gated(sets == 2)
    {
    }
    int64_t columns() const { return (int64_t)sets * half; }
    int64_t width() const { return (int64_t)sets * N; }
    bool padded() const { return half != N; }
};

size_t split_bytes(const ProductPlan &p, int64_t M, int64_t C)
{
    return p.splits > 1 ? align_up((size_t)p.splits * M * C * sizeof(float)) : 0;
}

// A product of tiles starts and ends in 3.4 us beside its steps; where N is no multiple
// of 8 it needs a padded copy of the weight first, and stores element by element (333
// rows, 416 terms, 1088 columns 4.9 us, 1085 columns 10.1).
struct ForwardLayout {
    RowsPlan rows;
    ProductPlan plan;
    size_t weight, partial, total;
    explicit ForwardLayout(const Sizes &z)
    {
        rows = plan_rows(z.M, z.K, z.N, z.sets);
        plan = ProductPlan{};
        weight = partial = total = 0;
        if (z.M <= 16)
            return;
        plan = plan_product(z.M, z.columns(), z.K, z.gated);
        const float copy = z.padded() ? 5.2f + (float)z.K * z.columns() * 4.0f / 5e6f : 0.0f;
        if (rows.mt > 0 && rows.us <= plan.us + 3.4f + copy)
            return;
        rows.mt = 0;
        partial = z.padded() ? align_up((size_t)z.K * z.columns() * 2) : 0;
        total = partial + split_bytes(plan, z.M, z.columns());
    }
};

// The two gradient products go together where that is estimated to take no longer than
// one after the other and a launch's 3 us: each takes the CUs that the other leaves idle
// (100 rows, 1024 terms, 512 columns 15.4 -> 9.5 us; 4096, 2048 and 1536
// 65 -> 53; 8192, 2048 and 1536 104 -> 98).
struct BackwardLayout {
    ProductPlan dx, dw;
    ProductPlan both_dx, both_dw;
    bool together;
    int strips;
    bool makes_dz;             // dz is not d_out as it is
    int parts;                 // bf16 values of one dz
    size_t weight, dz, bias, partial, total;
    explicit BackwardLayout(const Sizes &z, const moe_lora_linear_shape *s)
    {
        const int64_t M = std::max<int64_t>(z.M, 1);
        parts = s->out_fp32 ? 2 : 1;
        dx = plan_product(M, z.K, z.columns(), false, parts);
        dw = plan_product(z.K, z.columns(), M, false, parts);
        together = plan_both(M, z.K, z.columns(), parts, &both_dw, &both_dx) <= dx.us + dw.us + 3.0f;
        strips = act_grad_blocks(z.M);
        makes_dz = s->activation != MOE_LORA_ACT_NONE || s->out_fp32 || z.padded();
        size_t o = 0;
        auto take = [&](size_t bytes) {
            const size_t at = o;
            o += align_up(bytes);
            return at;
        };
        weight = take(z.padded() ? (size_t)z.K * z.columns() * 2 : 0);
        dz = take(makes_dz ? (size_t)z.M * z.columns() * 2 * parts : 0);
        bias = take((size_t)strips * z.width() * sizeof(float));
        // the two products run one after the other
        partial = take(std::max({split_bytes(dx, M, z.K), split_bytes(dw, z.K, z.columns()),
                                 together ? split_bytes(both_dw, z.K, z.columns()) : 0}));
        total = o;
    }
};

bool wide_epilogue(const Epilogue &e)
{
    return e.N % 8 == 0 && aligned(e.bias, 16) && aligned(e.residual, 16) && aligned(e.preact, 16) &&
           aligned(e.out, 16);
}

// ---- norms ----------------------------------------------------------------

int validate(const moe_lora_norm_shape *s)
{
    if (!s)
        return MOE_LORA_ERR_INVALID_ARG;
    if (s->rows < 0 || s->rows > 1 << 24 || s->hidden < 64 || s->hidden > 65536 || s->hidden % 64 != 0)
        return MOE_LORA_ERR_UNSUPPORTED_SHAPE;
    if (!(s->eps > 0.0f) || !std::isfinite(s->eps) || !std::isfinite(s->residual_scale) ||
        !std::isfinite(s->weight_offset))
        return MOE_LORA_ERR_INVALID_ARG;
    if (s->gate < MOE_LORA_GATE_NONE || s->gate > MOE_LORA_GATE_CHANNEL)
        return MOE_LORA_ERR_INVALID_ARG;
    return MOE_LORA_OK;
}

bool gate_aligned(const moe_lora_norm_shape *s, const void *gate)
{
    return aligned(gate, s->gate == MOE_LORA_GATE_TOKEN ? 4 : 16);
}

// ---- clipping -------------------------------------------------------------

constexpr int kMostTensors = 4096;
constexpr int64_t kMostElements = (int64_t)1 << 36;
constexpr int64_t kMostBlocks = 1 << 23;   // of a launch: its threads stay below 2^32

// Elements of a block: few values are spread over more blocks.
int chunk_of(const moe_lora_gradient *g, int32_t count)
{
    int64_t n = 0;
    for (int32_t i = 0; i < count; ++i)
        n += g[i].elements;
    int chunk = 2048;
    while (chunk < kClipLargest && n > chunk * (int64_t)1024)
        chunk *= 2;
    return chunk;
}

// More than the second-level caches hold (32 MB) is written past them: they and the last
// level then still have what the squares have read (60 tensors, 111 MB, in turn with
// others: 79.5 -> 68.5 us).  Less stays in them for its reader.
bool past_caches(const moe_lora_gradient *g, int32_t count)
{
    int64_t bytes = 0;
    for (int32_t i = 0; i < count; ++i)
        bytes += g[i].elements * (g[i].fp32 ? 4 : 2);
    return bytes > 32 << 20;
}

int64_t total_chunks(const moe_lora_gradient *g, int32_t count, int chunk)
{
    int64_t n = 0;
    for (int32_t i = 0; i < count; ++i)
        n += (g[i].elements + chunk - 1) / chunk;
    return n;
}

int validate(const moe_lora_gradient *g, int32_t count)
{
    if (count < 0 || count > kMostTensors)
        return MOE_LORA_ERR_UNSUPPORTED_SHAPE;
    if (count > 0 && !g)
        return MOE_LORA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < count; ++i) {
        if (g[i].elements < 0 || g[i].elements >= kMostElements)
            return MOE_LORA_ERR_UNSUPPORTED_SHAPE;
        if ((g[i].fp32 != 0 && g[i].fp32 != 1) || g[i].reserved != 0)
            return MOE_LORA_ERR_INVALID_ARG;
    }
    return MOE_LORA_OK;
}

struct Range {
    uintptr_t first, last;
};

// Range `which` of a table: the data of tensor which / 2, or its output (odd).
Range range_of(const moe_lora_gradient *g, int which)
{
    const moe_lora_gradient &t = g[which / 2];
    const uintptr_t first = reinterpret_cast<uintptr_t>(which & 1 ? t.out : t.data);
    return Range{first, first + (size_t)t.elements * (t.fp32 ? 4 : 2)};
}

// No range of one tensor meets one of another (a tensor's data and out are its own,
// and either the same or apart).  Two bytes of stack a range, and room for no more
// tensors than a call of that size needs: a caller's thread may have a small stack.
template <int TENSORS>
__attribute__((noinline)) bool ranges_apart(const moe_lora_gradient *g, int32_t count, bool scales)
{
    static_assert(2 * TENSORS <= 1 << 16, "indices are 16 bits");
    uint16_t order[2 * TENSORS];
    int n = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (g[i].elements == 0)
            continue;
        order[n++] = (uint16_t)(2 * i);
        if (scales && g[i].out != g[i].data)
            order[n++] = (uint16_t)(2 * i + 1);
    }
    auto before = [g](uint16_t a, uint16_t b) { return range_of(g, a).first < range_of(g, b).first; };
    if (!std::is_sorted(order, order + n, before))
        std::sort(order, order + n, before);
    for (int i = 1; i < n; ++i)
        if (range_of(g, order[i]).first < range_of(g, order[i - 1]).last)
            return false;
    return true;
}

// f(table, first chunk of the table) over the tensors with elements, as many to a
// table as fit
template <class F>
int for_tables(const moe_lora_gradient *g, int32_t count, int chunk, F f)
{
    ClipTable t;
    t.chunk = chunk;
    t.stream = past_caches(g, count);
    t.count = t.blocks = 0;
    int64_t done = 0;
    for (int32_t i = 0; i <= count; ++i) {
        const int64_t chunks = i < count ? (g[i].elements + chunk - 1) / chunk : 0;
        if (t.count > 0 && (i == count || t.count == kClipTensors || t.blocks + chunks > kMostBlocks)) {
            const hipError_t rc = f(t, done);
            if (rc != hipSuccess)
                return MOE_LORA_ERR_HIP;
            done += t.blocks;
            t.count = t.blocks = 0;
        }
        if (chunks > 0) {
            t.t[t.count++] = ClipTensor{g[i].data, g[i].out, g[i].elements, t.blocks, g[i].fp32};
            t.blocks += (int)chunks;
        }
    }
    return MOE_LORA_OK;
}

} // namespace

extern "C" {

size_t moe_lora_linear_workspace_size(const moe_lora_linear_shape *shape)
{
    return validate(shape) == MOE_LORA_OK ? ForwardLayout(Sizes(shape)).total : 0;
}

int moe_lora_linear(const moe_lora_linear_shape *shape, const void *x, const void *w, const float *bias,
                    const void *residual, void *out, void *preact, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    MOE_TRY(validate(shape));
    if (shape->rows == 0)
        return MOE_LORA_OK;
    if (!x || !w || !out)
        return MOE_LORA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 4) || !aligned(residual, 2) ||
        !aligned(out, shape->out_fp32 ? 4 : 2) || !aligned(preact, 2))
        return MOE_LORA_ERR_MISALIGNED;
    const Sizes z(shape);
    const ForwardLayout layout(z);
    MOE_TRY(check_workspace(workspace, workspace_bytes, layout.total));
    hipStream_t st = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    Epilogue e{};
    e.bias = bias;
    e.residual = static_cast<const uint16_t *>(residual);
    e.out = out;
    e.preact = static_cast<uint16_t *>(preact);
    e.N = e.half = z.N;
    e.sets = z.sets;
    e.act = shape->activation;
    e.fp32 = shape->out_fp32;
    e.wide = wide_epilogue(e);
    const auto *xp = static_cast<const uint16_t *>(x);
    const auto *wp = static_cast<const uint16_t *>(w);
    if (layout.rows.mt > 0)
        return check(launch_rows(layout.rows, RowsArgs{xp, wp, (int)z.M, (int)z.K, (int)z.width(), e}, st));
    if (z.padded()) {
        uint16_t *copy = reinterpret_cast<uint16_t *>(ws + layout.weight);
        MOE_TRY(check(launch_pad_columns(wp, copy, z.K, z.N, z.half, z.sets, st)));
        wp = copy;
        e.half = z.half;
    }
    ProductArgs a{};
    a.Q = xp;
    a.P = wp;
    a.M = (int)z.M;
    a.C = (int)z.columns();
    a.K = a.ldq = (int)z.K;
    a.ldp = a.C;
    a.partial = reinterpret_cast<float *>(ws + layout.partial);
    a.e = e;
    return check(launch_product(Product::forward, layout.plan, a, st));
}

size_t moe_lora_linear_backward_workspace_size(const moe_lora_linear_shape *shape)
{
    return validate(shape) == MOE_LORA_OK ? BackwardLayout(Sizes(shape), shape).total : 0;
}

int moe_lora_linear_backward(const moe_lora_linear_shape *shape, const void *x, const void *w,
                             const void *preact, const void *d_out, void *d_x, void *d_w, float *d_bias,
                             void *workspace, size_t workspace_bytes, void *stream)
{
    MOE_TRY(validate(shape));
    if (!d_x && !d_w && !d_bias)
        return MOE_LORA_ERR_INVALID_ARG;
    const bool act = shape->activation != MOE_LORA_ACT_NONE;
    if (shape->rows > 0 && (!d_out || (d_x && !w) || (d_w && !x) || (act && !preact)))
        return MOE_LORA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(d_x, 16) || !aligned(d_w, 16) || !aligned(d_bias, 4) ||
        !aligned(preact, 2) || !aligned(d_out, 16))
        return MOE_LORA_ERR_MISALIGNED;
    const Sizes z(shape);
    const BackwardLayout layout(z, shape);
    MOE_TRY(check_workspace(workspace, workspace_bytes, layout.total));
    hipStream_t st = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    const bool makes_dz = layout.makes_dz && (d_x || d_w);
    const uint16_t *dz = static_cast<const uint16_t *>(d_out);
    const int64_t part = layout.parts > 1 ? z.M * z.columns() : 0;
    if (makes_dz || d_bias) {
        ActGradArgs g{};
        g.d_out = d_out;
        g.preact = act ? static_cast<const uint16_t *>(preact) : nullptr;
        g.dz = makes_dz ? reinterpret_cast<uint16_t *>(ws + layout.dz) : nullptr;
        // one strip's sums are the sums
        g.partial = !d_bias ? nullptr : layout.strips == 1 ? d_bias : reinterpret_cast<float *>(ws + layout.bias);
        g.d_bias = d_bias;
        g.part = part;
        g.M = z.M;
        g.N = z.N;
        g.half = z.half;
        g.sets = z.sets;
        g.act = shape->activation;
        g.fp32 = shape->out_fp32;
        g.blocks = layout.strips;
        MOE_TRY(check(launch_act_grad(g, st)));
        if (makes_dz)
            dz = g.dz;
    }
    const auto *wp = static_cast<const uint16_t *>(w);
    float *partial = reinterpret_cast<float *>(ws + layout.partial);
    ProductArgs gw{}, gx{};
    if (d_w) {
        gw.Q = static_cast<const uint16_t *>(x);
        gw.P = dz;
        gw.M = gw.ldq = (int)z.K;
        gw.C = gw.ldp = (int)z.columns();
        gw.K = (int)z.M;
        gw.part = part;
        gw.partial = partial;
        gw.e.out = d_w;
        gw.e.N = z.padded() ? z.N : (int)z.columns();
        gw.e.half = z.half;
        gw.e.sets = z.sets;
        gw.e.padded = z.padded();
        gw.e.wide = wide_epilogue(gw.e);
    }
    if (d_x && z.M > 0) {
        if (z.padded()) {
            uint16_t *copy = reinterpret_cast<uint16_t *>(ws + layout.weight);
            MOE_TRY(check(launch_pad_columns(wp, copy, z.K, z.N, z.half, z.sets, st)));
            wp = copy;
        }
        gx.Q = dz;
        gx.P = wp;
        gx.M = (int)z.M;
        gx.C = (int)z.K;
        gx.K = gx.ldq = gx.ldp = (int)z.columns();
        gx.part = part;
        gx.partial = partial;
        gx.e.out = d_x;
        gx.e.N = gx.e.half = (int)z.K;
        gx.e.sets = 1;
        gx.e.wide = wide_epilogue(gx.e);
    }
    // together unless d_x overwrites x, which d_w reads: then d_w comes first
    if (gw.M > 0 && gx.M > 0 && d_x != x && layout.together)
        return check(launch_both_gradients(layout.both_dw, gw, layout.both_dx, gx, st));
    if (gw.M > 0)
        MOE_TRY(check(launch_product(Product::weight_grad, layout.dw, gw, st)));
    if (gx.M > 0)
        MOE_TRY(check(launch_product(Product::input_grad, layout.dx, gx, st)));
    return MOE_LORA_OK;
}

int moe_lora_block_norm(const moe_lora_norm_shape *shape, const void *residual, const void *branch,
                        const void *post_weight, const void *pre_weight, const void *gate,
                        void *new_residual, void *normed, void *stream)
{
    MOE_TRY(validate(shape));
    if (shape->rows == 0)
        return MOE_LORA_OK;
    if ((!residual && !branch) || (!new_residual && !normed) || (normed != nullptr) != (pre_weight != nullptr))
        return MOE_LORA_ERR_INVALID_ARG;
    if ((gate != nullptr) != (shape->gate != MOE_LORA_GATE_NONE) || (!branch && (post_weight || gate)))
        return MOE_LORA_ERR_INVALID_ARG;
    for (const void *p : {residual, branch, post_weight, pre_weight, (const void *)new_residual,
                          (const void *)normed})
        if (!aligned(p, 16))
            return MOE_LORA_ERR_MISALIGNED;
    if (!gate_aligned(shape, gate))
        return MOE_LORA_ERR_MISALIGNED;
    const NormArgs a{static_cast<const uint16_t *>(residual), static_cast<const uint16_t *>(branch),
                     static_cast<const uint16_t *>(post_weight), static_cast<const uint16_t *>(pre_weight),
                     gate, static_cast<uint16_t *>(new_residual), static_cast<uint16_t *>(normed),
                     shape->rows, shape->hidden, shape->gate, shape->eps, shape->residual_scale,
                     shape->weight_offset};
    return check(launch_block_norm(a, static_cast<hipStream_t>(stream)));
}

size_t moe_lora_block_norm_backward_workspace_size(const moe_lora_norm_shape *shape)
{
    if (validate(shape) != MOE_LORA_OK)
        return 0;
    return align_up(norm_grad_stats_bytes(shape->rows, shape->hidden)) +
           align_up((size_t)norm_grad_blocks(shape->rows, shape->hidden) * 3 * shape->hidden * sizeof(float));
}

int moe_lora_block_norm_backward(const moe_lora_norm_shape *shape, const void *new_residual,
                                 const void *branch, const void *post_weight, const void *pre_weight,
                                 const void *gate, const void *d_new_residual, const void *d_normed,
                                 const moe_lora_norm_gradients *gradients, void *workspace,
                                 size_t workspace_bytes, void *stream)
{
    MOE_TRY(validate(shape));
    if (!gradients)
        return MOE_LORA_ERR_INVALID_ARG;
    const moe_lora_norm_gradients &d = *gradients;
    if (!d.d_residual && !d.d_branch && !d.d_post_weight && !d.d_pre_weight && !d.d_gate)
        return MOE_LORA_ERR_INVALID_ARG;
    if ((gate != nullptr) != (shape->gate != MOE_LORA_GATE_NONE) || (d.d_gate && !gate) ||
        (d.d_post_weight && !post_weight))
        return MOE_LORA_ERR_INVALID_ARG;
    const bool some = shape->rows > 0;
    if (some) {
        if (!d_new_residual && !d_normed)
            return MOE_LORA_ERR_INVALID_ARG;
        if (d_normed ? !pre_weight || !new_residual : d.d_pre_weight != nullptr)
            return MOE_LORA_ERR_INVALID_ARG;
        if ((post_weight || d.d_gate) && !branch)
            return MOE_LORA_ERR_INVALID_ARG;
    }
    for (const void *p : {new_residual, branch, post_weight, pre_weight, d_new_residual, d_normed,
                          (const void *)d.d_residual, (const void *)d.d_branch})
        if (!aligned(p, 16))
            return MOE_LORA_ERR_MISALIGNED;
    if (!gate_aligned(shape, gate) || !aligned(d.d_post_weight, 4) || !aligned(d.d_pre_weight, 4) ||
        !aligned(d.d_gate, 4))
        return MOE_LORA_ERR_MISALIGNED;
    MOE_TRY(check_workspace(workspace, workspace_bytes, moe_lora_block_norm_backward_workspace_size(shape)));
    hipStream_t st = static_cast<hipStream_t>(stream);
    NormGradArgs a{};
    a.r = static_cast<const uint16_t *>(new_residual);
    a.y = static_cast<const uint16_t *>(branch);
    a.w_post = static_cast<const uint16_t *>(post_weight);
    a.w_pre = static_cast<const uint16_t *>(pre_weight);
    a.gate = gate;
    a.dr = static_cast<const uint16_t *>(d_new_residual);
    a.dz = static_cast<const uint16_t *>(d_normed);
    a.dx = static_cast<uint16_t *>(d.d_residual);
    a.dy = static_cast<uint16_t *>(d.d_branch);
    a.stats = static_cast<float4 *>(workspace);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                          align_up(norm_grad_stats_bytes(shape->rows, shape->hidden)));
    float *to[3];
    auto place = [&](float *out) {
        if (!out)
            return -1;
        to[a.sums] = out;
        return a.sums++;
    };
    a.post_at = place(d.d_post_weight);
    a.pre_at = place(d.d_pre_weight);
    a.gate_at = place(shape->gate == MOE_LORA_GATE_CHANNEL ? d.d_gate : nullptr);
    a.d_token = shape->gate == MOE_LORA_GATE_TOKEN ? d.d_gate : nullptr;
    a.T = shape->rows;
    a.H = shape->hidden;
    a.gate_kind = shape->gate;
    a.blocks = norm_grad_blocks(a.T, a.H);
    a.eps = shape->eps;
    a.alpha = shape->residual_scale;
    a.offset = shape->weight_offset;
    MOE_TRY(check(launch_block_norm_backward(a, st)));
    return a.sums > 0 ? check(launch_column_sums(a.partial, a.blocks, a.sums, a.H, to, st)) : MOE_LORA_OK;
}

size_t moe_lora_clip_workspace_size(const moe_lora_gradient *gradients, int32_t count)
{
    if (validate(gradients, count) != MOE_LORA_OK)
        return 0;
    return kAlign + align_up((size_t)total_chunks(gradients, count, chunk_of(gradients, count)) * sizeof(double));
}

int moe_lora_clip_gradients(const moe_lora_gradient *gradients, int32_t count, float max_norm,
                            float *norm, void *workspace, size_t workspace_bytes, void *stream)
{
    MOE_TRY(validate(gradients, count));
    if (!norm || !(max_norm >= 0.0f))
        return MOE_LORA_ERR_INVALID_ARG;
    if (!aligned(norm, 4))
        return MOE_LORA_ERR_MISALIGNED;
    const bool scales = !std::isinf(max_norm);
    for (int32_t i = 0; i < count; ++i) {
        const moe_lora_gradient &g = gradients[i];
        if (g.elements == 0)
            continue;
        if (!g.data || (scales && !g.out))
            return MOE_LORA_ERR_INVALID_ARG;
        const size_t size = g.fp32 ? 4 : 2;
        const uintptr_t data = reinterpret_cast<uintptr_t>(g.data), out = reinterpret_cast<uintptr_t>(g.out);
        if (data % size != 0 || (scales && out % size != 0))
            return MOE_LORA_ERR_MISALIGNED;
    }
    if (!(count <= 128 ? ranges_apart<128>(gradients, count, scales)
                       : ranges_apart<kMostTensors>(gradients, count, scales)))
        return MOE_LORA_ERR_INVALID_ARG;
    MOE_TRY(check_workspace(workspace, workspace_bytes, moe_lora_clip_workspace_size(gradients, count)));
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int chunk = chunk_of(gradients, count);
    const ClipSums c{reinterpret_cast<double *>(static_cast<char *>(workspace) + kAlign),
                     total_chunks(gradients, count, chunk), norm, static_cast<ClipFactor *>(workspace), max_norm};
    MOE_TRY(for_tables(gradients, count, chunk, [&](const ClipTable &t, int64_t done) {
        return launch_clip_squares(t, c.partial + done, st);
    }));
    if (!scales || c.blocks == 0 || c.blocks > kClipFew)
        MOE_TRY(check(launch_clip_norm(c, st)));
    if (!scales)
        return MOE_LORA_OK;
    return for_tables(gradients, count, chunk, [&](const ClipTable &t, int64_t done) {
        return launch_clip_scale(t, c, done == 0, st);
    });
}

} // extern "C"
