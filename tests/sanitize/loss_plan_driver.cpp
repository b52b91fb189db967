// Drives the loss operators' host layer (zero_loss_abi.cpp) with stub launchers
// under the sanitizers: distillation's entry points over random shapes, k and strides,
// and of every plan the tiles, the slabs' room and the launches that the kernels derive
// from it.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>

#include "zero_launch.h"
#include "zero_loss.h"
#include "zero_loss_launch.h"

static zloss::Call last;
namespace zloss {
const char* launch_loss(const Call& c, void*) { last = c; return nullptr; }
const char* launch_grad(const Call& c, void*) { last = c; return nullptr; }
}  // namespace zloss
namespace zlaunch {
const char* launch_step(const StepArgs&, void*) { return nullptr; }
const char* launch_init(const InitArgs&, void*) { return nullptr; }
const char* launch_step_mean(const StepArgs&, void*) { return nullptr; }
const char* launch_mean(const MeanArgs&, void*) { return nullptr; }
int64_t mean_partials(int, int64_t) { return 1; }
const char* launch_sumsq_finalize(const double*, int64_t, double*, void*) { return nullptr; }
const char* stream_wait(void*, void*) { return nullptr; }
const char* scratch_address(void*, double** o) { *o = nullptr; return nullptr; }
}  // namespace zlaunch

static int failures = 0;
#define CHECK(x) \
  do { \
    if (!(x)) { ++failures; std::printf("FAILED %s:%d %s\n", __FILE__, __LINE__, #x); } \
  } while (0)

static int64_t over(int64_t x, int64_t m) { return (x + m - 1) / m; }

// What zero_loss.hip makes of a plan: tiles, their threads, slabs.
static void check_plan(const zloss::Plan& q, const zero_head& h, int64_t gathered) {
  const bool few = h.tokens <= zloss::kFewTokens;
  CHECK(q.tile_m == 256 || q.tile_m == 128);
  CHECK(q.tile_n == 64 || (q.tile_n == 256 && q.tile_m == 256));
  // few tokens: only 64 rows of hidden and of the rows' parameters are packed
  CHECK(!few || q.tile_n == 64);
  CHECK(q.rows % q.tile_n == 0 && q.piece % q.tile_m == 0);
  CHECK(q.planes == (h.dtype == ZERO_LOSS_F32 ? 3 : 1));
  const int64_t threads = q.tile_n == 256 ? 512 : q.tile_m == 256 ? 256 : 128;
  const int64_t rows = std::min(q.piece, q.vocab);
  const int64_t blocks =
      over(over(rows, q.tile_m) * over(q.rows, q.tile_n), 8) * 8 + over(gathered, 16) * 8;
  CHECK(blocks * threads < (INT64_C(1) << 32));
  if (!q.grad) return;
  const int64_t across = over(q.dimp, 256), tile_rows = few ? 64 : 256;
  const int64_t tiles = over(std::max<int64_t>(h.tokens, 1), tile_rows) * across;
  CHECK(tiles <= q.acc_tiles);
  CHECK(q.o_acc + (size_t)q.acc_tiles * tile_rows * 256 * 4 <= q.total);
  // one slab of the sum fits its tiles
  CHECK(h.tokens * q.dimp <= tiles * tile_rows * 256);
  const int64_t w_tiles = over(rows, few ? 128 : 256) * over(q.dimp, few ? 128 : 256);
  const int64_t d_tiles = std::max<int64_t>(few ? 0 : q.rows / 256 * across, q.acc_tiles);
  CHECK((w_tiles + d_tiles + 16) * 512 < (INT64_C(1) << 32));
}

int main() {
  std::mt19937_64 rng(11);
  const auto pick = [&](double lo, double hi) {  // spread over the logarithm
    return (int64_t)std::exp2(
        std::uniform_real_distribution<double>(std::log2(lo), std::log2(hi))(rng));
  };
  char* base = reinterpret_cast<char*>(UINT64_C(0x100000000000));
  const auto at = [&](int i) { return base + (int64_t)i * (INT64_C(1) << 44); };
  const auto fat = [&](int i) { return reinterpret_cast<float*>(at(i)); };
  for (int i = 0; i < 20000; ++i) {
    zero_head h{};
    h.tokens = i % 50 == 0 ? 0 : i % 3 ? pick(1, ZERO_LOSS_MAX_TOKENS + 1) : pick(1, 100);
    if (i % 97 == 0) h.tokens = ZERO_LOSS_MAX_TOKENS;
    h.vocab = i % 89 == 0 ? ZERO_LOSS_MAX_VOCAB : pick(1, ZERO_LOSS_MAX_VOCAB + 1);
    h.dim = i % 83 == 0 ? ZERO_LOSS_MAX_DIM : pick(1, ZERO_LOSS_MAX_DIM + 1);
    if (i % 2) h.dim = (h.dim + 63) / 64 * 64;
    h.dtype = (int32_t)(rng() % 3);
    const int64_t es = h.dtype == ZERO_LOSS_F32 ? 4 : 2;
    h.hidden = at(0);
    h.hidden_stride = h.dim + pick(1, 100) - 1;
    h.weight = at(1) + (i % 5 == 0 ? es : 0);
    h.weight_stride = h.dim + (i % 3 ? 0 : pick(1, 100));
    zero_distill_params p{};
    p.index = at(2);
    p.logit = at(3);
    p.k = (int32_t)pick(1, ZERO_LOSS_MAX_K + 1);
    p.index_stride = p.k + (i % 4 ? 0 : pick(1, 1000));
    p.logit_stride = p.k + (i % 7 ? 0 : pick(1, 1000));
    p.index_dtype = i & 1;
    p.logit_dtype = (int32_t)(rng() % 3);
    p.temperature = 0.25 * (double)pick(1, 64);
    const int64_t ies = p.index_dtype == ZERO_INDEX_I64 ? 8 : 4;
    const int64_t les = p.logit_dtype == ZERO_LOSS_F32 ? 4 : 2;
    zero_head_grads g{};
    g.upstream = fat(4);
    g.upstream_stride = i & 1;
    g.dhidden = at(5);
    g.dhidden_stride = h.dim;
    g.dweight = at(6) + es;
    g.dweight_stride = h.dim + 3;
    size_t need[2] = {0, 0};
    CHECK(zero_loss_workspace_bytes(&h, 0, &need[0]) == ZERO_OK);
    CHECK(zero_loss_workspace_bytes(&h, 1, &need[1]) == ZERO_OK);
    // the loss, with its outputs anywhere
    const auto loss = [&](float* l, float* z, float* kept, size_t n) {
      return zero_linear_distill(&h, &p, l, z, kept, at(10), n, nullptr);
    };
    const auto grad = [&](size_t n) {
      return zero_linear_distill_grad(&h, &p, fat(8), fat(9), &g, at(10), n, nullptr);
    };
    CHECK(loss(fat(7), fat(8), fat(9), need[0]) == ZERO_OK);
    if (h.tokens > 0) {
      const int64_t waves = h.tokens * over(p.k, 16);
      CHECK(last.k == p.k && last.index_stride == p.index_stride);
      check_plan(last.plan, h, h.tokens <= zloss::kFewTokens ? waves : 0);
      CHECK(loss(fat(7), fat(8), fat(9), need[0] - 1) == ZERO_EINVAL);
      // an output on the last entry of a strided input, and just behind it
      const int64_t iend = (h.tokens - 1) * p.index_stride * ies + p.k * ies;
      const int64_t lend = (h.tokens - 1) * p.logit_stride * les + p.k * les;
      CHECK(loss((float*)(at(2) + (iend - 1) / 4 * 4), fat(8), fat(9), need[0]) == ZERO_EINVAL);
      CHECK(loss((float*)(at(2) + over(iend, 4) * 4), fat(8), fat(9), need[0]) == ZERO_OK);
      CHECK(loss(fat(7), (float*)(at(3) + (lend - 1) / 4 * 4), fat(9), need[0]) == ZERO_EINVAL);
      CHECK(loss(fat(7), (float*)(at(3) + over(lend, 4) * 4), fat(9), need[0]) == ZERO_OK);
      CHECK(loss(fat(9) + h.tokens * p.k - 1, fat(8), fat(9), need[0]) == ZERO_EINVAL);
      CHECK(loss(fat(9) + h.tokens * p.k, fat(8), fat(9), need[0]) == ZERO_OK);
    }
    CHECK(grad(need[1]) == ZERO_OK);
    CHECK(last.logit_in == fat(9) && last.lse_in == fat(8));
    check_plan(last.plan, h, 0);
    CHECK(grad(need[1] - 1) == ZERO_EINVAL);
    if (h.tokens > 0) {
      // a gradient on the last saved logit
      g.dweight = fat(9) + h.tokens * p.k - 1;
      CHECK(grad(need[1]) == ZERO_EINVAL);
      g.dweight = fat(9) + h.tokens * p.k;
      CHECK(grad(need[1]) == ZERO_OK);
    }
  }
  std::printf("loss plans: %d failures\n", failures);
  return failures != 0;
}
