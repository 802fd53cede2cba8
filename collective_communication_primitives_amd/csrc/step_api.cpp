// step_api.cpp -- the C ABI of the model-step operators of include/dt.h:
// argument checks, row tables and workspace sizes.  The arithmetic is in
// norm.hip, moe.hip and loss.hip; nothing here allocates or throws.
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>

#include "dt.h"
#include "dt_step.h"

static_assert(sizeof(dt::NormBackArgs) <= 4096, "kernel arguments must stay below 4 KiB");
static_assert(sizeof(dt::ExchangeRowsArgs) <= 4096, "kernel arguments must stay below 4 KiB");

namespace {

using dt::RowTable;

dt_status fail(dt_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return dt::report_error(st, buf);
}

dt_status done(hipError_t e, const char* what) {
    if (e == hipSuccess) return DT_OK;
    return fail(DT_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

dt_status check_ranks(int nranks) {
    if (nranks < 1 || nranks > DT_MAX_RANKS)
        return fail(DT_ERR_ARG, "nranks=%d outside [1, %d]", nranks, DT_MAX_RANKS);
    return DT_OK;
}

dt_status check_float(dt_dtype d, const char* what) {
    if (d == DT_FLOAT32 || d == DT_BFLOAT16) return DT_OK;
    if (d == DT_INT32) return fail(DT_ERR_UNSUPPORTED, "%s takes fp32 or bf16, not int32", what);
    return fail(DT_ERR_ARG, "bad dtype %d", int(d));
}

size_t esize_of(dt_dtype d) { return d == DT_BFLOAT16 ? 2 : 4; }

// The ranks' row counts as a table of first rows.
dt_status row_table(const size_t* counts, int nranks, const char* name, RowTable& t) {
    if (counts == nullptr) return fail(DT_ERR_ARG, "%s is NULL", name);
    uint64_t sum = 0;
    for (int r = 0; r <= DT_MAX_RANKS; r++) t.start[r] = 0;
    for (int r = 0; r < nranks; r++) {
        if (counts[r] >= DT_MAX_STEP_ROWS || (sum += counts[r]) >= DT_MAX_STEP_ROWS)
            return fail(DT_ERR_ARG, "%s: %d or more rows in all", name, DT_MAX_STEP_ROWS);
        t.start[r + 1] = uint32_t(sum);
    }
    for (int r = nranks; r < DT_MAX_RANKS; r++) t.start[r + 1] = uint32_t(sum);
    return DT_OK;
}

// The byte ranges one call reads and writes: every buffer checked for NULL
// and element alignment, and no written range may meet another range.
class Ranges {
  public:
    // Buffer `index` of `list`, n bytes of elements of `align` bytes; empty
    // buffers may be NULL.
    template <typename P>
    void add(P const* list, int index, size_t n, size_t align, bool write, const char* name) {
        if (st_ != DT_OK) return;
        if (list == nullptr) {
            st_ = fail(DT_ERR_ARG, "%s is NULL", name);
            return;
        }
        if (n == 0) return;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(list[index]);
        if (lo == 0) st_ = fail(DT_ERR_ARG, "%s[%d] is NULL", name, index);
        else if (lo % align != 0) st_ = fail(DT_ERR_ARG, "%s[%d] is not aligned to its elements", name, index);
        else r_[n_++] = Range{lo, lo + n, name, index, write};
    }
    dt_status check(const char* what) {
        if (st_ != DT_OK) return st_;
        std::sort(r_, r_ + n_, [](const Range& a, const Range& b) { return a.lo < b.lo; });
        const Range* any = nullptr;      // the range, and the written one, that reach furthest so far
        const Range* written = nullptr;
        for (int i = 0; i < n_; i++) {
            const Range& x = r_[i];
            const Range* hit = x.write ? any : written;
            if (hit != nullptr && x.lo < hit->hi)
                return fail(DT_ERR_ARG, "%s: %s[%d] and %s[%d] overlap", what, hit->name, hit->index, x.name, x.index);
            if (any == nullptr || x.hi > any->hi) any = &x;
            if (x.write && (written == nullptr || x.hi > written->hi)) written = &x;
        }
        return DT_OK;
    }

  private:
    struct Range {
        uintptr_t lo, hi;
        const char* name;
        int index;
        bool write;
    };
    Range r_[12 * DT_MAX_RANKS];
    int n_ = 0;
    dt_status st_ = DT_OK;
};

// A list of per-rank pointers copied into kernel arguments (NULL list: all NULL).
template <typename D, typename S>
void copy_list(D (&to)[dt::kMaxRanksHost], S const* from, int nranks) {
    for (int r = 0; r < dt::kMaxRanksHost; r++) to[r] = from != nullptr && r < nranks ? from[r] : nullptr;
}

dt_status check_workspace(const void* ws, size_t have, size_t need, const char* what) {
    if (need == 0) return DT_OK;
    if (ws == nullptr || have < need)
        return fail(DT_ERR_ARG, "%s needs %zu bytes of workspace, got %zu", what, need, ws == nullptr ? size_t(0) : have);
    if (reinterpret_cast<uintptr_t>(ws) % 256 != 0) return fail(DT_ERR_ARG, "%s: workspace must be 256-byte aligned", what);
    return DT_OK;
}

dt_status check_cols(size_t cols, const char* what) {
    if (cols < 1 || cols > DT_MAX_STEP_COLS)
        return fail(DT_ERR_ARG, "%s: cols=%zu outside [1, %d]", what, cols, DT_MAX_STEP_COLS);
    return DT_OK;
}

// A launch of the expert calls takes up to 256 threads a token, and HIP counts
// a launch's threads in 32 bits.
dt_status check_tokens(const RowTable& t, int nranks) {
    if (t.start[nranks] > DT_MAX_MOE_TOKENS)
        return fail(DT_ERR_ARG, "tokens: %u in all, above %d", t.start[nranks], DT_MAX_MOE_TOKENS);
    return DT_OK;
}

dt_status check_experts(int nexperts, int topk) {
    if (nexperts < 1 || nexperts > DT_MAX_EXPERTS)
        return fail(DT_ERR_ARG, "nexperts=%d outside [1, %d]", nexperts, DT_MAX_EXPERTS);
    if (topk < 1 || topk > nexperts || topk > DT_MAX_TOPK)
        return fail(DT_ERR_ARG, "topk=%d outside [1, min(nexperts, %d)]", topk, DT_MAX_TOPK);
    return DT_OK;
}

#define TRY(expr)                                \
    do {                                         \
        const dt_status try_st = (expr);         \
        if (try_st != DT_OK) return try_st;      \
    } while (0)

}  // namespace

extern "C" {

// -------------------------------------------------------------- layer norm --
size_t dt_layer_norm_workspace(int nranks, const size_t* rows, size_t cols) {
    RowTable t;
    dt::report_error(DT_OK, "");
    if (check_ranks(nranks) != DT_OK || row_table(rows, nranks, "rows", t) != DT_OK ||
        check_cols(cols, "layer_norm_workspace") != DT_OK)
        return 0;
    return size_t(dt::norm_strips(t.start[nranks], uint32_t(cols))) * 2 * cols * sizeof(float);
}

dt_status dt_layer_norm(const void* const* x, const void* const* weight, const void* const* bias, void* const* y,
                        float* const* mean, float* const* rstd, int nranks, const size_t* rows, size_t cols, float eps,
                        dt_dtype dtype, hipStream_t stream) {
    dt::report_error(DT_OK, "");
    dt::NormArgs a = {};
    TRY(check_ranks(nranks));
    TRY(check_float(dtype, "layer_norm"));
    TRY(row_table(rows, nranks, "rows", a.rows));
    TRY(check_cols(cols, "layer_norm"));
    if (!(eps >= 0.f) || eps > 1e30f) return fail(DT_ERR_ARG, "layer_norm: eps must be finite and not negative");
    if ((mean == nullptr) != (rstd == nullptr)) return fail(DT_ERR_ARG, "layer_norm: mean and rstd come together");
    const size_t es = esize_of(dtype);
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        const size_t n = rows[r] * cols * es;
        g.add(x, r, n, es, false, "x");
        g.add(y, r, n, es, true, "y");
        if (rows[r] > 0) {
            g.add(weight, r, cols * es, es, false, "weight");
            if (bias != nullptr) g.add(bias, r, cols * es, es, false, "bias");
        }
        if (mean != nullptr) {
            g.add(mean, r, rows[r] * sizeof(float), sizeof(float), true, "mean");
            g.add(rstd, r, rows[r] * sizeof(float), sizeof(float), true, "rstd");
        }
    }
    TRY(g.check("layer_norm"));
    if (a.rows.start[nranks] == 0) return DT_OK;
    copy_list(a.x, x, nranks);
    copy_list(a.weight, weight, nranks);
    copy_list(a.bias, bias, nranks);
    copy_list(a.y, y, nranks);
    copy_list(a.mean, mean, nranks);
    copy_list(a.rstd, rstd, nranks);
    a.cols = uint32_t(cols);
    a.eps = eps;
    a.nranks = nranks;
    return done(dt::launch_norm(a, dtype, stream), "layer_norm");
}

dt_status dt_layer_norm_backward(const void* const* dy, const void* const* x, const void* const* weight,
                                 const float* const* mean, const float* const* rstd, void* const* dx,
                                 void* const* dweight, void* const* dbias, int nranks, const size_t* rows, size_t cols,
                                 dt_dtype dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    dt::report_error(DT_OK, "");
    dt::NormBackArgs a = {};
    TRY(check_ranks(nranks));
    TRY(check_float(dtype, "layer_norm_backward"));
    TRY(row_table(rows, nranks, "rows", a.rows));
    TRY(check_cols(cols, "layer_norm_backward"));
    const size_t es = esize_of(dtype);
    a.strips = dt::norm_strips(a.rows.start[nranks], uint32_t(cols));
    const size_t need = size_t(a.strips) * 2 * cols * sizeof(float);
    TRY(check_workspace(workspace, workspace_bytes, need, "layer_norm_backward"));
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        const size_t n = rows[r] * cols * es;
        g.add(dy, r, n, es, false, "dy");
        g.add(x, r, n, es, false, "x");
        g.add(dx, r, n, es, true, "dx");
        if (rows[r] > 0) g.add(weight, r, cols * es, es, false, "weight");
        g.add(mean, r, rows[r] * sizeof(float), sizeof(float), false, "mean");
        g.add(rstd, r, rows[r] * sizeof(float), sizeof(float), false, "rstd");
        g.add(dweight, r, cols * es, es, true, "dweight");
        if (dbias != nullptr) g.add(dbias, r, cols * es, es, true, "dbias");
    }
    g.add(&workspace, 0, need, 1, true, "workspace");
    TRY(g.check("layer_norm_backward"));
    copy_list(a.dy, dy, nranks);
    copy_list(a.x, x, nranks);
    copy_list(a.weight, weight, nranks);
    copy_list(a.mean, mean, nranks);
    copy_list(a.rstd, rstd, nranks);
    copy_list(a.dx, dx, nranks);
    copy_list(a.dweight, dweight, nranks);
    copy_list(a.dbias, dbias, nranks);
    a.partial = static_cast<float*>(workspace);
    a.cols = uint32_t(cols);
    a.nranks = nranks;
    return done(dt::launch_norm_backward(a, dtype, stream), "layer_norm_backward");
}

// ----------------------------------------------------------------- routing --
dt_status dt_moe_route(const void* const* logits, int32_t* const* experts, float* const* weights, int nranks,
                       const size_t* tokens, int nexperts, int topk, const float* bias, int groups, int topk_groups,
                       dt_score score, int renormalize, float scale, dt_dtype dtype, hipStream_t stream) {
    dt::report_error(DT_OK, "");
    dt::RouteArgs a = {};
    TRY(check_ranks(nranks));
    TRY(check_float(dtype, "moe_route"));
    TRY(row_table(tokens, nranks, "tokens", a.rows));
    TRY(check_tokens(a.rows, nranks));
    TRY(check_experts(nexperts, topk));
    if (score != DT_SCORE_SOFTMAX && score != DT_SCORE_SIGMOID) return fail(DT_ERR_ARG, "bad score %d", int(score));
    if (groups < 1 || groups > DT_MAX_GROUPS || nexperts % groups != 0)
        return fail(DT_ERR_ARG, "groups=%d must divide nexperts=%d and be at most %d", groups, nexperts, DT_MAX_GROUPS);
    if (topk_groups < 1 || topk_groups > groups || topk > nexperts / groups * topk_groups)
        return fail(DT_ERR_ARG, "topk_groups=%d of %d groups cannot hold topk=%d", topk_groups, groups, topk);
    const size_t es = esize_of(dtype);
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        g.add(logits, r, tokens[r] * nexperts * es, es, false, "logits");
        g.add(experts, r, tokens[r] * topk * sizeof(int32_t), sizeof(int32_t), true, "experts");
        g.add(weights, r, tokens[r] * topk * sizeof(float), sizeof(float), true, "weights");
    }
    if (bias != nullptr) g.add(&bias, 0, nexperts * sizeof(float), sizeof(float), false, "bias");
    TRY(g.check("moe_route"));
    if (a.rows.start[nranks] == 0) return DT_OK;
    copy_list(a.logits, logits, nranks);
    copy_list(a.experts, experts, nranks);
    copy_list(a.weights, weights, nranks);
    a.bias = bias;
    a.nexperts = uint32_t(nexperts);
    a.topk = uint32_t(topk);
    a.groups = uint32_t(groups);
    // every group stays: the choice is that without groups
    if (topk_groups == groups) a.groups = 1;
    a.topk_groups = uint32_t(topk_groups);
    a.sigmoid = score == DT_SCORE_SIGMOID;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    return done(dt::launch_route(a, nranks, dtype, stream), "moe_route");
}

dt_status dt_moe_route_backward(const void* const* logits, const int32_t* const* experts, const float* const* dweights,
                                void* const* dlogits, int nranks, const size_t* tokens, int nexperts, int topk,
                                dt_score score, int renormalize, float scale, dt_dtype dtype, hipStream_t stream) {
    dt::report_error(DT_OK, "");
    dt::RouteBackArgs a = {};
    TRY(check_ranks(nranks));
    TRY(check_float(dtype, "moe_route_backward"));
    TRY(row_table(tokens, nranks, "tokens", a.rows));
    TRY(check_tokens(a.rows, nranks));
    TRY(check_experts(nexperts, topk));
    if (score != DT_SCORE_SOFTMAX && score != DT_SCORE_SIGMOID) return fail(DT_ERR_ARG, "bad score %d", int(score));
    const size_t es = esize_of(dtype);
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        g.add(logits, r, tokens[r] * nexperts * es, es, false, "logits");
        g.add(experts, r, tokens[r] * topk * sizeof(int32_t), sizeof(int32_t), false, "experts");
        g.add(dweights, r, tokens[r] * topk * sizeof(float), sizeof(float), false, "dweights");
        g.add(dlogits, r, tokens[r] * nexperts * es, es, true, "dlogits");
    }
    TRY(g.check("moe_route_backward"));
    if (a.rows.start[nranks] == 0) return DT_OK;
    copy_list(a.logits, logits, nranks);
    copy_list(a.experts, experts, nranks);
    copy_list(a.dweights, dweights, nranks);
    copy_list(a.dlogits, dlogits, nranks);
    a.nexperts = uint32_t(nexperts);
    a.topk = uint32_t(topk);
    a.sigmoid = score == DT_SCORE_SIGMOID;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    return done(dt::launch_route_backward(a, nranks, dtype, stream), "moe_route_backward");
}

}  // extern "C"

// ---------------------------------------------------------------- exchange --
namespace {

struct ExchangeShape {
    RowTable rows;
    uint32_t capacity[dt::kMaxRanksHost];
    uint32_t per_rank;
};

dt_status exchange_shape(int nranks, const size_t* tokens, const size_t* capacity, size_t cols, int nexperts, int topk,
                         const char* what, ExchangeShape& s) {
    TRY(check_ranks(nranks));
    TRY(row_table(tokens, nranks, "tokens", s.rows));
    TRY(check_cols(cols, what));
    TRY(check_experts(nexperts, topk));
    if (nexperts % nranks != 0) return fail(DT_ERR_ARG, "%s: %d experts do not divide by %d ranks", what, nexperts, nranks);
    if (uint64_t(s.rows.start[nranks]) * topk >= DT_MAX_STEP_ROWS)
        return fail(DT_ERR_ARG, "%s: %d or more slots in all", what, DT_MAX_STEP_ROWS);
    TRY(check_tokens(s.rows, nranks));
    if (capacity == nullptr) return fail(DT_ERR_ARG, "capacity is NULL");
    for (int q = 0; q < nranks; q++) {
        if (capacity[q] >= DT_MAX_STEP_ROWS) return fail(DT_ERR_ARG, "capacity[%d] is too large", q);
        s.capacity[q] = uint32_t(capacity[q]);
    }
    s.per_rank = uint32_t(nexperts / nranks);
    return DT_OK;
}

void fill_exchange(dt::ExchangeRowsArgs& a, const ExchangeShape& s, int nranks, size_t cols, int nexperts, int topk) {
    a.rows = s.rows;
    for (int q = 0; q < nranks; q++) a.capacity[q] = s.capacity[q];
    a.cols = uint32_t(cols);
    a.nexperts = uint32_t(nexperts);
    a.topk = uint32_t(topk);
    a.per_rank = s.per_rank;
    a.nranks = nranks;
}

size_t plan_bytes(const RowTable& rows, int nranks, int nexperts, int topk) {
    return size_t(dt::plan_blocks(uint64_t(rows.start[nranks]) * topk) + 1) * nexperts * sizeof(uint32_t);
}

}  // namespace

extern "C" {

size_t dt_moe_dispatch_workspace(int nranks, const size_t* tokens, int nexperts, int topk) {
    RowTable t;
    dt::report_error(DT_OK, "");
    if (check_ranks(nranks) != DT_OK || row_table(tokens, nranks, "tokens", t) != DT_OK ||
        check_tokens(t, nranks) != DT_OK || check_experts(nexperts, topk) != DT_OK)
        return 0;
    return plan_bytes(t, nranks, nexperts, topk);
}

dt_status dt_moe_dispatch(const void* const* x, const int32_t* const* experts, void* const* recv,
                          int32_t* const* positions, int32_t* const* offsets, int nranks, const size_t* tokens,
                          const size_t* capacity, size_t cols, int nexperts, int topk, dt_dtype dtype, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
    dt::report_error(DT_OK, "");
    ExchangeShape s;
    TRY(exchange_shape(nranks, tokens, capacity, cols, nexperts, topk, "moe_dispatch", s));
    if (dtype != DT_FLOAT32 && dtype != DT_BFLOAT16 && dtype != DT_INT32) return fail(DT_ERR_ARG, "bad dtype %d", int(dtype));
    const size_t es = esize_of(dtype);
    const size_t need = plan_bytes(s.rows, nranks, nexperts, topk);
    TRY(check_workspace(workspace, workspace_bytes, need, "moe_dispatch"));
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        g.add(x, r, tokens[r] * cols * es, es, false, "x");
        g.add(experts, r, tokens[r] * topk * sizeof(int32_t), sizeof(int32_t), false, "experts");
        g.add(recv, r, capacity[r] * cols * es, es, true, "recv");
        g.add(positions, r, tokens[r] * topk * sizeof(int32_t), sizeof(int32_t), true, "positions");
        g.add(offsets, r, (s.per_rank + 1) * sizeof(int32_t), sizeof(int32_t), true, "offsets");
    }
    g.add(&workspace, 0, need, 1, true, "workspace");
    TRY(g.check("moe_dispatch"));
    dt::PlanArgs p = {};
    copy_list(p.experts, experts, nranks);
    copy_list(p.positions, positions, nranks);
    copy_list(p.offsets, offsets, nranks);
    for (int q = 0; q < nranks; q++) p.capacity[q] = s.capacity[q];
    p.rows = s.rows;
    p.counts = static_cast<uint32_t*>(workspace);
    p.nexperts = uint32_t(nexperts);
    p.topk = uint32_t(topk);
    p.per_rank = s.per_rank;
    p.nranks = nranks;
    dt::ExchangeRowsArgs a = {};
    fill_exchange(a, s, nranks, cols, nexperts, topk);
    copy_list(a.tokens_in, x, nranks);
    copy_list(a.rows_out, recv, nranks);
    copy_list(a.experts, experts, nranks);
    copy_list(a.positions, positions, nranks);
    return done(dt::launch_dispatch(p, a, int(es), stream), "moe_dispatch");
}

dt_status dt_moe_combine(const void* const* y, const int32_t* const* experts, const int32_t* const* positions,
                         const float* const* weights, void* const* out, int nranks, const size_t* tokens,
                         const size_t* capacity, size_t cols, int nexperts, int topk, dt_dtype dtype,
                         hipStream_t stream) {
    dt::report_error(DT_OK, "");
    ExchangeShape s;
    TRY(exchange_shape(nranks, tokens, capacity, cols, nexperts, topk, "moe_combine", s));
    TRY(check_float(dtype, "moe_combine"));
    const size_t es = esize_of(dtype);
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        const size_t slots = tokens[r] * topk;
        g.add(y, r, capacity[r] * cols * es, es, false, "y");
        g.add(experts, r, slots * sizeof(int32_t), sizeof(int32_t), false, "experts");
        g.add(positions, r, slots * sizeof(int32_t), sizeof(int32_t), false, "positions");
        if (weights != nullptr) g.add(weights, r, slots * sizeof(float), sizeof(float), false, "weights");
        g.add(out, r, tokens[r] * cols * es, es, true, "out");
    }
    TRY(g.check("moe_combine"));
    if (s.rows.start[nranks] == 0) return DT_OK;
    dt::ExchangeRowsArgs a = {};
    fill_exchange(a, s, nranks, cols, nexperts, topk);
    copy_list(a.rows_in, y, nranks);
    copy_list(a.experts, experts, nranks);
    copy_list(a.positions, positions, nranks);
    copy_list(a.weights, weights, nranks);
    copy_list(a.tokens_out, out, nranks);
    return done(dt::launch_combine(a, dtype, stream), "moe_combine");
}

dt_status dt_moe_combine_backward(const void* const* dout, const void* const* y, const int32_t* const* experts,
                                  const int32_t* const* positions, const float* const* weights, void* const* dy,
                                  float* const* dweights, int nranks, const size_t* tokens, const size_t* capacity,
                                  size_t cols, int nexperts, int topk, dt_dtype dtype, hipStream_t stream) {
    dt::report_error(DT_OK, "");
    ExchangeShape s;
    TRY(exchange_shape(nranks, tokens, capacity, cols, nexperts, topk, "moe_combine_backward", s));
    TRY(check_float(dtype, "moe_combine_backward"));
    const size_t es = esize_of(dtype);
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        const size_t slots = tokens[r] * topk;
        g.add(dout, r, tokens[r] * cols * es, es, false, "dout");
        g.add(y, r, capacity[r] * cols * es, es, false, "y");
        g.add(experts, r, slots * sizeof(int32_t), sizeof(int32_t), false, "experts");
        g.add(positions, r, slots * sizeof(int32_t), sizeof(int32_t), false, "positions");
        g.add(weights, r, slots * sizeof(float), sizeof(float), false, "weights");
        g.add(dy, r, capacity[r] * cols * es, es, true, "dy");
        g.add(dweights, r, slots * sizeof(float), sizeof(float), true, "dweights");
    }
    TRY(g.check("moe_combine_backward"));
    if (s.rows.start[nranks] == 0) return DT_OK;
    dt::ExchangeRowsArgs a = {};
    fill_exchange(a, s, nranks, cols, nexperts, topk);
    copy_list(a.tokens_in, dout, nranks);
    copy_list(a.rows_in, y, nranks);
    copy_list(a.rows_out, dy, nranks);
    copy_list(a.experts, experts, nranks);
    copy_list(a.positions, positions, nranks);
    copy_list(a.weights, weights, nranks);
    copy_list(a.dweights, dweights, nranks);
    return done(dt::launch_combine_backward(a, dtype, stream), "moe_combine_backward");
}

}  // extern "C"

// --------------------------------------------------------- vocabulary loss --
namespace {

dt_status loss_shape(int nranks, const size_t* vocab_rows, size_t tokens, size_t cols, dt_dtype dtype, const char* what,
                     RowTable& t) {
    TRY(check_ranks(nranks));
    TRY(check_float(dtype, what));
    TRY(row_table(vocab_rows, nranks, "vocab_rows", t));
    TRY(check_cols(cols, what));
    if (t.start[nranks] == 0) return fail(DT_ERR_ARG, "%s: the vocabulary is empty", what);
    if (tokens > DT_MAX_LOSS_TOKENS) return fail(DT_ERR_ARG, "%s: tokens=%zu above %d", what, tokens, DT_MAX_LOSS_TOKENS);
    return DT_OK;
}

}  // namespace

extern "C" {

size_t dt_vocab_loss_workspace(int nranks, const size_t* vocab_rows, size_t tokens, size_t cols, dt_dtype dtype) {
    RowTable t;
    dt::report_error(DT_OK, "");
    if (loss_shape(nranks, vocab_rows, tokens, cols, dtype, "vocab_loss_workspace", t) != DT_OK) return 0;
    return dt::loss_workspace(t, nranks, tokens, cols, dtype);
}

dt_status dt_vocab_loss(const void* const* hidden, const void* const* weight, const int64_t* const* targets,
                        float* const* loss, float* const* lse, int nranks, const size_t* vocab_rows, size_t tokens,
                        size_t cols, int64_t ignore_index, dt_dtype dtype, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
    dt::report_error(DT_OK, "");
    dt::LossArgs a = {};
    TRY(loss_shape(nranks, vocab_rows, tokens, cols, dtype, "vocab_loss", a.vocab));
    const size_t es = esize_of(dtype);
    const size_t need = dt::loss_workspace(a.vocab, nranks, tokens, cols, dtype);
    TRY(check_workspace(workspace, workspace_bytes, need, "vocab_loss"));
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        g.add(hidden, r, tokens * cols * es, es, false, "hidden");
        g.add(weight, r, vocab_rows[r] * cols * es, es, false, "weight");
        g.add(targets, r, tokens * sizeof(int64_t), sizeof(int64_t), false, "targets");
        g.add(loss, r, tokens * sizeof(float), sizeof(float), true, "loss");
        g.add(lse, r, tokens * sizeof(float), sizeof(float), true, "lse");
    }
    g.add(&workspace, 0, need, 1, true, "workspace");
    TRY(g.check("vocab_loss"));
    if (tokens == 0) return DT_OK;
    a.hidden = hidden[0];
    copy_list(a.weight, weight, nranks);
    a.targets = targets[0];
    copy_list(a.loss, loss, nranks);
    copy_list(a.lse, lse, nranks);
    a.tokens = uint32_t(tokens);
    a.cols = uint32_t(cols);
    a.ignore_index = ignore_index;
    a.workspace = static_cast<char*>(workspace);
    a.nranks = nranks;
    return done(dt::launch_loss(a, dtype, stream), "vocab_loss");
}

size_t dt_vocab_loss_backward_workspace(int nranks, const size_t* vocab_rows, size_t tokens, size_t cols,
                                        size_t piece_rows, dt_dtype dtype) {
    RowTable t;
    dt::report_error(DT_OK, "");
    if (loss_shape(nranks, vocab_rows, tokens, cols, dtype, "vocab_loss_backward_workspace", t) != DT_OK) return 0;
    const uint32_t piece = dt::loss_piece(t, nranks, tokens, cols, dtype, piece_rows);
    return dt::loss_backward_workspace(nranks, tokens, cols, piece, dtype);
}

dt_status dt_vocab_loss_backward(const void* const* hidden, const void* const* weight, const int64_t* const* targets,
                                 const float* const* lse, const float* const* dloss, void* const* dhidden,
                                 void* const* dweight, int nranks, const size_t* vocab_rows, size_t tokens, size_t cols,
                                 int64_t ignore_index, size_t piece_rows, dt_dtype dtype, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    dt::report_error(DT_OK, "");
    dt::LossArgs a = {};
    TRY(loss_shape(nranks, vocab_rows, tokens, cols, dtype, "vocab_loss_backward", a.vocab));
    const size_t es = esize_of(dtype);
    a.piece = dt::loss_piece(a.vocab, nranks, tokens, cols, dtype, piece_rows);
    const size_t need = dt::loss_backward_workspace(nranks, tokens, cols, a.piece, dtype);
    TRY(check_workspace(workspace, workspace_bytes, need, "vocab_loss_backward"));
    Ranges g;
    for (int r = 0; r < nranks; r++) {
        g.add(hidden, r, tokens * cols * es, es, false, "hidden");
        g.add(weight, r, vocab_rows[r] * cols * es, es, false, "weight");
        g.add(targets, r, tokens * sizeof(int64_t), sizeof(int64_t), false, "targets");
        g.add(lse, r, tokens * sizeof(float), sizeof(float), false, "lse");
        g.add(dloss, r, tokens * sizeof(float), sizeof(float), false, "dloss");
        g.add(dhidden, r, tokens * cols * es, es, true, "dhidden");
        g.add(dweight, r, vocab_rows[r] * cols * es, es, true, "dweight");
    }
    g.add(&workspace, 0, need, 1, true, "workspace");
    TRY(g.check("vocab_loss_backward"));
    a.hidden = hidden[0];
    copy_list(a.weight, weight, nranks);
    a.targets = targets[0];
    a.lse_in = lse[0];
    a.dloss = dloss[0];
    copy_list(a.dhidden, dhidden, nranks);
    copy_list(a.dweight, dweight, nranks);
    a.tokens = uint32_t(tokens);
    a.cols = uint32_t(cols);
    a.ignore_index = ignore_index;
    a.workspace = static_cast<char*>(workspace);
    a.nranks = nranks;
    return done(dt::launch_loss_backward(a, dtype, stream), "vocab_loss_backward");
}

}  // extern "C"
