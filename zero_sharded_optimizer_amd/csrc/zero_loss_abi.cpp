// Host side of the C ABI declared in include/zero_loss.h: argument validation,
// the pieces of the vocabulary and the workspace layout. Touches no HIP API;
// device work goes through zloss::.
#include "zero_loss.h"

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "zero_error.h"
#include "zero_loss_launch.h"

namespace {

using zerror::fail;
using zerror::ok;

static_assert((int)ZERO_LOSS_F32 == (int)zloss::kF32 && (int)ZERO_LOSS_BF16 == (int)zloss::kBF16 &&
                  (int)ZERO_LOSS_F16 == (int)zloss::kF16,
              "zero_loss_dtype and zloss::Dtype must agree");

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t ceil_div(int64_t x, int64_t m) { return (x + m - 1) / m; }

int64_t dtype_size(int32_t d) { return d == ZERO_LOSS_F32 ? 4 : 2; }
int64_t index_size(int32_t d) { return d == ZERO_INDEX_I64 ? 8 : 4; }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A two-dimensional region: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Region {
  uintptr_t lo;
  int64_t rows, width, pitch;
  const char* name;
  uintptr_t hi() const {
    return rows > 0 && width > 0 ? lo + (uintptr_t)((rows - 1) * pitch + width) : lo;
  }
};

// Whether two regions share a byte. Two column ranges of one pitched buffer
// (the same pitch) interleave without sharing any; other interleavings are
// taken as sharing.
bool shares(const Region& x, const Region& y) {
  if (x.lo >= x.hi() || y.lo >= y.hi() || x.lo >= y.hi() || y.lo >= x.hi()) return false;
  if (x.pitch != y.pitch || x.pitch <= 0) return true;
  const int64_t p = x.pitch;
  const int64_t d = (int64_t)(((y.lo - x.lo) % (uintptr_t)p + (uintptr_t)p) % (uintptr_t)p);
  if (x.lo > y.lo) {
    const int64_t e = (int64_t)((x.lo - y.lo) % (uintptr_t)p);
    return !(e >= y.width && e + x.width <= p);
  }
  return !(d >= x.width && d + y.width <= p);
}

zero_status check_head(const zero_head* h) {
  if (h == nullptr) return fail(ZERO_EINVAL, "head is NULL");
  if (h->reserved != 0) return fail(ZERO_EINVAL, "head.reserved must be 0");
  if (h->dtype < ZERO_LOSS_F32 || h->dtype > ZERO_LOSS_F16)
    return fail(ZERO_EINVAL, "unknown head.dtype %d", h->dtype);
  if (h->tokens < 0 || h->tokens > ZERO_LOSS_MAX_TOKENS)
    return fail(ZERO_EINVAL, "tokens must be in [0, %d], got %lld", ZERO_LOSS_MAX_TOKENS,
                (long long)h->tokens);
  if (h->vocab < 1 || h->vocab > ZERO_LOSS_MAX_VOCAB)
    return fail(ZERO_EINVAL, "vocab must be in [1, %d], got %lld", ZERO_LOSS_MAX_VOCAB,
                (long long)h->vocab);
  if (h->dim < 1 || h->dim > ZERO_LOSS_MAX_DIM)
    return fail(ZERO_EINVAL, "dim must be in [1, %d], got %lld", ZERO_LOSS_MAX_DIM,
                (long long)h->dim);
  constexpr int64_t kMaxStride = INT64_C(1) << 32;
  if (h->hidden_stride < h->dim || h->hidden_stride > kMaxStride)
    return fail(ZERO_EINVAL, "hidden_stride must be in [dim, 2^32]");
  if (h->weight_stride < h->dim || h->weight_stride > kMaxStride)
    return fail(ZERO_EINVAL, "weight_stride must be in [dim, 2^32]");
  if (h->weight == nullptr) return fail(ZERO_EINVAL, "weight is NULL");
  if (h->hidden == nullptr && h->tokens > 0) return fail(ZERO_EINVAL, "hidden is NULL");
  const uintptr_t es = (uintptr_t)dtype_size(h->dtype);
  if (!aligned(h->hidden, es) || !aligned(h->weight, es))
    return fail(ZERO_EINVAL, "hidden and weight must be aligned to their element size");
  return ZERO_OK;
}

// Vocabulary rows per piece. The largest allowed has 512 MiB of g, or of packed
// weights, or 2048 rows where those are more (g: beyond 2^17 tokens, some 43000 in fp32;
// 4 GiB at 2^20 tokens, 12 GiB in fp32). 256 MiB, what the chip's last cache holds, is
// 0.5 to 3% slower for the larger problems: dhidden's sum is then read and written more
// often; 128 MiB is another 1 to 7%. Smaller pieces are taken where the rounds of 256
// tiles that the chip holds at once come out fuller, in all: the logits' tiles [piece,
// tokens] take dim / 64 steps each, dweight's [dim, piece] tokens / 64, either about four
// steps more, and a piece about eight in launches. (dhidden's tiles fill up dweight's
// last round.)
int64_t choose_piece(const zloss::Plan& p, int64_t whole) {
  constexpr int64_t kPieceBytes = INT64_C(512) << 20;
  int64_t most = std::min<int64_t>(whole, INT64_C(1) << 21);
  most = std::min(most, (INT64_C(1) << 38) / p.rows);
  if (p.grad) most = std::min(most, kPieceBytes / (p.rows * 2 * p.planes));
  if (p.pack_w) most = std::min(most, kPieceBytes / (p.dimp * 2 * p.planes));
  most = std::max<int64_t>(most / zloss::kVocPad * zloss::kVocPad, std::min<int64_t>(whole, 2048));
  const int64_t least = ceil_div(whole, most);
  int64_t best = most, best_cost = INT64_MAX;
  for (int64_t n = least; n <= least + 8; ++n) {
    const int64_t piece = round_up(ceil_div(p.vocab, n), zloss::kVocPad);
    int64_t cost = 0;
    for (int64_t v0 = 0; v0 < p.vocab; v0 += piece) {
      const int64_t m = ceil_div(std::min(piece, p.vocab - v0), 256);
      cost += 8 + ceil_div(m * (p.rows / 256), 256) * (p.dimp / 64 + 4);
      const int64_t across = ceil_div(p.dimp, 256);
      if (p.grad)
        cost += (m * across * (p.rows / 64 + 4) + p.rows / 256 * across * (m * 4 + 32)) / 256 + 16;
    }
    if (cost < best_cost) {
      best = piece;
      best_cost = cost;
    }
  }
  return best;
}

// The logits' tiles. A compute unit holds one of 256 x 256, two of 256 x 64 or three
// of 128 x 64. The large one does most per byte it copies; the others are for
// problems with fewer large tiles than the chip has units, and for few tokens, whose
// logits are the weight's way from memory: more units read, and end together. Times
// of a round of `held` tiles, and of a last one that gives each unit but one or two,
// in microseconds a step and at the end, as measured (200 tokens x 5000 x 2048: 44, 29
// and 24 us in this order; 200 x 32000 x 2048: 45, 40, 53; 500 x 32000 x 2048: 56, 74,
// 88; 40 x 50257 x 4096: -, 72, 80).
void choose_tile(zloss::Plan* p) {
  struct Kind {
    int m, n, held;
    double step[3], more;  // by how many tiles the busiest unit has
  };
  static constexpr Kind kinds[3] = {{256, 256, 256, {1.35, 1.35, 1.35}, 6},
                                    {256, 64, 512, {0.85, 1.15, 1.15}, 3},
                                    {128, 64, 768, {0.70, 0.92, 1.05}, 3}};
  const int64_t rows = std::min(p->piece, p->vocab);
  const double steps = (double)(p->dimp / 64) * (p->planes > 1 ? 6 : 1);
  double best = HUGE_VAL;
  for (const Kind& k : kinds) {
    if (k.n == 256 && p->tokens <= zloss::kFewTokens) continue;
    const int64_t tiles = ceil_div(rows, k.m) * ceil_div(std::max<int64_t>(p->tokens, 1), k.n);
    const int64_t full = tiles / k.held, rest = tiles % k.held;
    const int last = k.held / 256 - 1;
    double cost = (double)full * (k.step[last] * steps + k.more);
    if (rest > 0) cost += k.step[std::min<int64_t>((rest - 1) / 256, last)] * steps + k.more;
    if (cost < best) {
      best = cost;
      p->tile_m = k.m;
      p->tile_n = k.n;
    }
  }
}

// The pieces and the workspace of one call.
zloss::Plan make_plan(const zero_head& h, bool grad) {
  zloss::Plan p{};
  p.tokens = h.tokens;
  p.vocab = h.vocab;
  p.dim = h.dim;
  p.dtype = h.dtype;
  p.planes = h.dtype == ZERO_LOSS_F32 ? 3 : 1;
  p.grad = grad;
  p.rows = round_up(std::max<int64_t>(h.tokens, 1), zloss::kRowPad);
  p.dimp = round_up(h.dim, zloss::kDimPad);
  // The tiles load 16 bytes a lane along a row and step over whole multiples of
  // kDimPad; lane offsets within 256 rows are 32-bit.
  p.pack_w = p.planes > 1 || p.dimp != h.dim || h.weight_stride % 8 != 0 ||
             h.weight_stride > (INT64_C(1) << 22) || !aligned(h.weight, 16);
  const int64_t whole = round_up(h.vocab, zloss::kVocPad);
  // The loss of unpacked weights stores nothing of a piece; but one launch has at
  // most 2^22 tiles (2^31 work-items, of the 2^32 that it could describe).
  p.piece = std::min(whole, (INT64_C(1) << 38) / p.rows / zloss::kVocPad * zloss::kVocPad);
  if (grad || p.pack_w) p.piece = choose_piece(p, whole);
  choose_tile(&p);
  p.stat_cols = whole / zloss::kStatRows;
  // dhidden's sum over the vocabulary may be cut into slabs, as long as they are
  // at most this many tiles of 256 columns, and of 256 tokens or 64.
  const int64_t tile_rows = h.tokens <= zloss::kFewTokens ? 64 : 256;
  const int64_t tiles = ceil_div(std::max<int64_t>(h.tokens, 1), tile_rows) * ceil_div(p.dimp, 256);
  p.acc_tiles = (int)std::max<int64_t>(512, tiles);

  size_t at = 0;
  const auto take = [&at](int64_t bytes) {
    const size_t o = at;
    at += (size_t)round_up(bytes, 256);
    return o;
  };
  p.o_head = take(256);
  p.o_rowmap = take(p.rows * 4);
  p.o_pos = take(p.rows * 4);
  p.o_state = take(p.rows);
  p.o_h = take(p.planes * p.rows * p.dimp * 2);
  p.o_w = take(p.pack_w ? p.planes * p.piece * p.dimp * 2 : 0);
  if (!grad) {
    p.o_stat = take(p.rows * p.stat_cols * 8);
    p.o_sum = take(p.rows * p.stat_cols * 4);
    p.o_entry = take(p.rows * 4);
  } else {
    p.o_rowp = take(p.rows * 32);
    p.o_g = take(p.planes * p.rows * p.piece * 2);
    p.o_acc = take(p.acc_tiles * tile_rows * 256 * 4);
  }
  p.total = at;
  return p;
}

zero_status check_workspace(const zloss::Plan& p, void* ws, size_t bytes) {
  if (ws == nullptr) return fail(ZERO_EINVAL, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(ZERO_EINVAL, "workspace must be 256-byte aligned");
  if (bytes < p.total)
    return fail(ZERO_EINVAL, "workspace holds %zu bytes, the call needs %zu", bytes, p.total);
  return ZERO_OK;
}

zero_status check_floats(const void* p, const char* name) {
  if (p == nullptr) return fail(ZERO_EINVAL, "%s is NULL", name);
  if (!aligned(p, 4)) return fail(ZERO_EINVAL, "%s must be 4-byte aligned", name);
  return ZERO_OK;
}

// The regions of one call: none of the first n_out may share a byte with any other.
struct Regions {
  Region r[16];
  int n = 0, n_out = 0;
  void add(const void* p, int64_t rows, int64_t width, int64_t pitch, const char* name) {
    if (p != nullptr) r[n++] = {(uintptr_t)p, rows, width, pitch, name};
  }
  void outputs_end() { n_out = n; }
  zero_status check() const {
    for (int i = 0; i < n_out; ++i)
      for (int j = 0; j < n; ++j)
        if (i != j && shares(r[i], r[j]))
          return fail(ZERO_EINVAL, "%s overlaps %s", r[i].name, r[j].name);
    return ZERO_OK;
  }
};

void head_regions(const zero_head& h, Regions* rg) {
  const int64_t es = dtype_size(h.dtype);
  rg->add(h.hidden, h.tokens, h.dim * es, h.hidden_stride * es, "hidden");
  rg->add(h.weight, h.vocab, h.dim * es, h.weight_stride * es, "weight");
}

void fill_head(const zero_head& h, const zloss::Plan& plan, void* ws, zloss::Call* c) {
  *c = zloss::Call{};
  c->plan = plan;
  c->hidden = h.hidden;
  c->hidden_stride = h.hidden_stride;
  c->weight = h.weight;
  c->weight_stride = h.weight_stride;
  c->ws = static_cast<char*>(ws);
  c->temperature = 1.0f;
}

zero_status check_xent(const zero_head& h, const zero_xent_params* p) {
  if (p == nullptr) return fail(ZERO_EINVAL, "params is NULL");
  if (p->reserved != 0) return fail(ZERO_EINVAL, "params.reserved must be 0");
  if (p->index_dtype != ZERO_INDEX_I32 && p->index_dtype != ZERO_INDEX_I64)
    return fail(ZERO_EINVAL, "unknown index_dtype %d", p->index_dtype);
  if (p->target == nullptr && h.tokens > 0) return fail(ZERO_EINVAL, "target is NULL");
  if (!aligned(p->target, (uintptr_t)index_size(p->index_dtype)))
    return fail(ZERO_EINVAL, "target must be aligned to its element size");
  if (!(p->label_smoothing >= 0.0 && (float)p->label_smoothing < 1.0f))
    return fail(ZERO_EINVAL, "label_smoothing must be in [0, 1) (as a float)");
  if (!(std::isfinite((float)p->z_loss) && p->z_loss >= 0.0))
    return fail(ZERO_EINVAL, "z_loss must be finite (as a float) and >= 0");
  return ZERO_OK;
}

void fill_xent(const zero_xent_params& p, zloss::Call* c) {
  c->target = p.target;
  c->index64 = p.index_dtype == ZERO_INDEX_I64;
  c->ignore_index = p.ignore_index;
  c->smoothing = (float)p.label_smoothing;
  c->z_loss = (float)p.z_loss;
  c->k = 0;
}

zero_status check_distill(const zero_head& h, const zero_distill_params* p) {
  if (p == nullptr) return fail(ZERO_EINVAL, "params is NULL");
  if (p->reserved != 0) return fail(ZERO_EINVAL, "params.reserved must be 0");
  if (p->k < 1 || p->k > ZERO_LOSS_MAX_K)
    return fail(ZERO_EINVAL, "k must be in [1, %d], got %d", ZERO_LOSS_MAX_K, p->k);
  if (p->index_dtype != ZERO_INDEX_I32 && p->index_dtype != ZERO_INDEX_I64)
    return fail(ZERO_EINVAL, "unknown index_dtype %d", p->index_dtype);
  if (p->logit_dtype < ZERO_LOSS_F32 || p->logit_dtype > ZERO_LOSS_F16)
    return fail(ZERO_EINVAL, "unknown logit_dtype %d", p->logit_dtype);
  constexpr int64_t kMaxStride = INT64_C(1) << 32;
  if (p->index_stride < p->k || p->index_stride > kMaxStride || p->logit_stride < p->k ||
      p->logit_stride > kMaxStride)
    return fail(ZERO_EINVAL, "index_stride and logit_stride must be in [k, 2^32]");
  if ((p->index == nullptr || p->logit == nullptr) && h.tokens > 0)
    return fail(ZERO_EINVAL, "index or logit is NULL");
  if (!aligned(p->index, (uintptr_t)index_size(p->index_dtype)) ||
      !aligned(p->logit, (uintptr_t)dtype_size(p->logit_dtype)))
    return fail(ZERO_EINVAL, "index and logit must be aligned to their element size");
  // What the kernels form of it, as floats: its square, and log2(e) over it, which lies
  // further from either end of the range.
  const float t = (float)p->temperature;
  if (!(t > 0.0f && std::isnormal(t * t)))
    return fail(ZERO_EINVAL, "temperature must be > 0, its square (as floats) neither infinite "
                             "nor subnormal");
  return ZERO_OK;
}

void fill_distill(const zero_distill_params& p, zloss::Call* c) {
  c->target = p.index;
  c->index64 = p.index_dtype == ZERO_INDEX_I64;
  c->k = p.k;
  c->index_stride = p.index_stride;
  c->logit_stride = p.logit_stride;
  c->teacher = p.logit;
  c->teacher_dtype = p.logit_dtype;
  c->temperature = (float)p.temperature;
}

zero_status check_grads(const zero_head& h, const zero_head_grads* g) {
  if (g == nullptr) return fail(ZERO_EINVAL, "grads is NULL");
  if (g->dhidden == nullptr && g->dweight == nullptr)
    return fail(ZERO_EINVAL, "dhidden and dweight are both NULL");
  if (h.tokens > 0) {
    const zero_status s = check_floats(g->upstream, "upstream");
    if (s != ZERO_OK) return s;
  }
  constexpr int64_t kMaxStride = INT64_C(1) << 32;
  if (g->upstream_stride < 0 || g->upstream_stride > kMaxStride)
    return fail(ZERO_EINVAL, "upstream_stride must be in [0, 2^32]");
  const uintptr_t es = (uintptr_t)dtype_size(h.dtype);
  if (!aligned(g->dhidden, es) || !aligned(g->dweight, es))
    return fail(ZERO_EINVAL, "dhidden and dweight must be aligned to their element size");
  if (g->dhidden != nullptr && (g->dhidden_stride < h.dim || g->dhidden_stride > kMaxStride))
    return fail(ZERO_EINVAL, "dhidden_stride must be in [dim, 2^32]");
  if (g->dweight != nullptr && (g->dweight_stride < h.dim || g->dweight_stride > kMaxStride))
    return fail(ZERO_EINVAL, "dweight_stride must be in [dim, 2^32]");
  return ZERO_OK;
}

void grad_outputs(const zero_head& h, const zero_head_grads& g, Regions* rg) {
  const int64_t es = dtype_size(h.dtype);
  rg->add(g.dhidden, h.tokens, h.dim * es, g.dhidden_stride * es, "dhidden");
  rg->add(g.dweight, h.vocab, h.dim * es, g.dweight_stride * es, "dweight");
}

void grad_inputs(const zero_head& h, const zero_head_grads& g, const float* lse, Regions* rg) {
  if (h.tokens > 0)
    rg->add(g.upstream, 1, ((h.tokens - 1) * g.upstream_stride + 1) * 4, 0, "upstream");
  rg->add(lse, 1, h.tokens * 4, 0, "lse");
}

void fill_grads(const zero_head_grads& g, const float* lse, zloss::Call* c) {
  c->lse_in = lse;
  c->upstream = g.upstream;
  c->upstream_stride = g.upstream_stride;
  c->dhidden = g.dhidden;
  c->dhidden_stride = g.dhidden_stride;
  c->dweight = g.dweight;
  c->dweight_stride = g.dweight_stride;
}

zero_status run(const char* err, const char* what) {
  if (err != nullptr) return fail(ZERO_EHIP, "%s launch failed: %s", what, err);
  return ok();
}

}  // namespace

extern "C" {

zero_status zero_loss_workspace_bytes(const zero_head* head, int32_t want_grad, size_t* bytes) {
  const zero_status s = check_head(head);
  if (s != ZERO_OK) return s;
  if (bytes == nullptr) return fail(ZERO_EINVAL, "bytes is NULL");
  *bytes = make_plan(*head, want_grad != 0).total;
  return ok();
}

zero_status zero_linear_xent(const zero_head* head, const zero_xent_params* p, float* loss,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  zero_status s = check_head(head);
  if (s != ZERO_OK) return s;
  if ((s = check_xent(*head, p)) != ZERO_OK) return s;
  const int64_t T = head->tokens;
  if (T == 0) return ok();  // no row: no buffer is touched
  if ((s = check_floats(loss, "loss")) != ZERO_OK) return s;
  if ((s = check_floats(lse, "lse")) != ZERO_OK) return s;
  const zloss::Plan plan = make_plan(*head, false);
  if ((s = check_workspace(plan, workspace, workspace_bytes)) != ZERO_OK) return s;
  Regions rg;
  rg.add(loss, 1, T * 4, 0, "loss");
  rg.add(lse, 1, T * 4, 0, "lse");
  rg.add(workspace, 1, (int64_t)plan.total, 0, "workspace");
  rg.outputs_end();
  head_regions(*head, &rg);
  rg.add(p->target, 1, T * index_size(p->index_dtype), 0, "target");
  if ((s = rg.check()) != ZERO_OK) return s;
  zloss::Call c;
  fill_head(*head, plan, workspace, &c);
  fill_xent(*p, &c);
  c.loss = loss;
  c.lse = lse;
  return run(zloss::launch_loss(c, stream), "xent");
}

zero_status zero_linear_xent_grad(const zero_head* head, const zero_xent_params* p,
                                  const float* lse, const zero_head_grads* grads, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  zero_status s = check_head(head);
  if (s != ZERO_OK) return s;
  if ((s = check_xent(*head, p)) != ZERO_OK) return s;
  if ((s = check_grads(*head, grads)) != ZERO_OK) return s;
  const int64_t T = head->tokens;
  if (T > 0 && (s = check_floats(lse, "lse")) != ZERO_OK) return s;
  const zloss::Plan plan = make_plan(*head, true);
  if ((s = check_workspace(plan, workspace, workspace_bytes)) != ZERO_OK) return s;
  Regions rg;
  grad_outputs(*head, *grads, &rg);
  rg.add(workspace, 1, (int64_t)plan.total, 0, "workspace");
  rg.outputs_end();
  head_regions(*head, &rg);
  rg.add(p->target, 1, T * index_size(p->index_dtype), 0, "target");
  grad_inputs(*head, *grads, lse, &rg);
  if ((s = rg.check()) != ZERO_OK) return s;
  zloss::Call c;
  fill_head(*head, plan, workspace, &c);
  fill_xent(*p, &c);
  fill_grads(*grads, lse, &c);
  return run(zloss::launch_grad(c, stream), "xent gradient");
}

zero_status zero_linear_distill(const zero_head* head, const zero_distill_params* p, float* loss,
                                float* lse, float* logit, void* workspace, size_t workspace_bytes,
                                void* stream) {
  zero_status s = check_head(head);
  if (s != ZERO_OK) return s;
  if ((s = check_distill(*head, p)) != ZERO_OK) return s;
  const int64_t T = head->tokens;
  if (T == 0) return ok();  // no row: no buffer is touched
  if ((s = check_floats(loss, "loss")) != ZERO_OK) return s;
  if ((s = check_floats(lse, "lse")) != ZERO_OK) return s;
  if ((s = check_floats(logit, "logit")) != ZERO_OK) return s;
  const zloss::Plan plan = make_plan(*head, false);
  if ((s = check_workspace(plan, workspace, workspace_bytes)) != ZERO_OK) return s;
  Regions rg;
  rg.add(loss, 1, T * 4, 0, "loss");
  rg.add(lse, 1, T * 4, 0, "lse");
  rg.add(logit, 1, T * p->k * 4, 0, "logit");
  rg.add(workspace, 1, (int64_t)plan.total, 0, "workspace");
  rg.outputs_end();
  head_regions(*head, &rg);
  rg.add(p->index, T, p->k * index_size(p->index_dtype),
         p->index_stride * index_size(p->index_dtype), "params.index");
  rg.add(p->logit, T, p->k * dtype_size(p->logit_dtype),
         p->logit_stride * dtype_size(p->logit_dtype), "params.logit");
  if ((s = rg.check()) != ZERO_OK) return s;
  zloss::Call c;
  fill_head(*head, plan, workspace, &c);
  fill_distill(*p, &c);
  c.loss = loss;
  c.lse = lse;
  c.logit = logit;
  return run(zloss::launch_loss(c, stream), "distill");
}

zero_status zero_linear_distill_grad(const zero_head* head, const zero_distill_params* p,
                                     const float* lse, const float* logit,
                                     const zero_head_grads* grads, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  zero_status s = check_head(head);
  if (s != ZERO_OK) return s;
  if ((s = check_distill(*head, p)) != ZERO_OK) return s;
  if ((s = check_grads(*head, grads)) != ZERO_OK) return s;
  const int64_t T = head->tokens;
  if (T > 0 && (s = check_floats(lse, "lse")) != ZERO_OK) return s;
  if (T > 0 && (s = check_floats(logit, "logit")) != ZERO_OK) return s;
  const zloss::Plan plan = make_plan(*head, true);
  if ((s = check_workspace(plan, workspace, workspace_bytes)) != ZERO_OK) return s;
  Regions rg;
  grad_outputs(*head, *grads, &rg);
  rg.add(workspace, 1, (int64_t)plan.total, 0, "workspace");
  rg.outputs_end();
  head_regions(*head, &rg);
  rg.add(p->index, T, p->k * index_size(p->index_dtype),
         p->index_stride * index_size(p->index_dtype), "params.index");
  rg.add(p->logit, T, p->k * dtype_size(p->logit_dtype),
         p->logit_stride * dtype_size(p->logit_dtype), "params.logit");
  grad_inputs(*head, *grads, lse, &rg);
  rg.add(logit, 1, T * p->k * 4, 0, "logit");
  if ((s = rg.check()) != ZERO_OK) return s;
  zloss::Call c;
  fill_head(*head, plan, workspace, &c);
  fill_distill(*p, &c);
  fill_grads(*grads, lse, &c);
  c.logit_in = logit;
  return run(zloss::launch_grad(c, stream), "distill gradient");
}

}  // extern "C"
