// Drives the loss operators' host layer (zero_loss_abi.cpp) with stub launchers
// under the sanitizers: refusals, and the pieces and workspace layout over random
// shapes, with the properties the kernels rely on.
#include <cstdint>
#include <cmath>
#include <cstdio>
#include <cstdlib>
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

int main() {
  std::mt19937_64 rng(7);
  const auto pick = [&](double lo, double hi) {  // spread over the logarithm
    return (int64_t)std::exp2(std::uniform_real_distribution<double>(std::log2(lo), std::log2(hi))(rng));
  };
  char* base = reinterpret_cast<char*>(UINT64_C(0x100000000000));
  const auto at = [&](int i) { return base + (int64_t)i * (INT64_C(1) << 44); };
  for (int i = 0; i < 20000; ++i) {
    zero_head h{};
    h.tokens = i % 50 == 0 ? 0 : pick(1, ZERO_LOSS_MAX_TOKENS + 1);
    h.vocab = pick(1, ZERO_LOSS_MAX_VOCAB + 1);
    h.dim = pick(1, ZERO_LOSS_MAX_DIM + 1);
    if (i % 2) h.dim = (h.dim + 63) / 64 * 64;
    h.dtype = i % 3;
    const int64_t es = h.dtype == ZERO_LOSS_F32 ? 4 : 2;
    h.hidden = at(0);
    h.hidden_stride = h.dim + pick(1, 100) - 1;
    h.weight = at(1) + (i % 5 == 0 ? es : 0);
    h.weight_stride = h.dim + (i % 3 ? 0 : pick(1, 100));
    zero_xent_params p{};
    p.target = at(2);
    p.index_dtype = i & 1;
    zero_head_grads g{};
    g.upstream = reinterpret_cast<float*>(at(3));
    g.upstream_stride = i & 1;
    g.dhidden = at(4);
    g.dhidden_stride = h.dim;
    g.dweight = at(5) + es;
    g.dweight_stride = h.dim + 3;
    size_t fwd = 0, bwd = 0;
    CHECK(zero_loss_workspace_bytes(&h, 0, &fwd) == ZERO_OK);
    CHECK(zero_loss_workspace_bytes(&h, 1, &bwd) == ZERO_OK);
    float* f = reinterpret_cast<float*>(at(6));
    for (int grad = 0; grad < 2; ++grad) {
      const size_t need = grad ? bwd : fwd;
      const auto call = [&](size_t n) {
        return grad ? zero_linear_xent_grad(&h, &p, f, &g, at(7), n, nullptr)
                    : zero_linear_xent(&h, &p, f, reinterpret_cast<float*>(at(8)), at(7), n,
                                       nullptr);
      };
      if (grad || h.tokens > 0) CHECK(call(need - 1) == ZERO_EINVAL);
      CHECK(call(need) == ZERO_OK);
      if (!grad && h.tokens == 0) continue;
      const zloss::Plan& q = last.plan;
      CHECK(q.rows % 256 == 0 && q.rows >= h.tokens && q.rows < h.tokens + 257);
      CHECK(q.dimp % 64 == 0 && q.dimp >= h.dim);
      CHECK(q.pack_w || (q.dimp == h.dim && h.weight_stride % 8 == 0 &&
                         reinterpret_cast<uintptr_t>(h.weight) % 16 == 0));
      CHECK(q.piece % 256 == 0 && q.piece >= 256);
      CHECK(q.rows / 256 * (q.piece / 256) <= (INT64_C(1) << 22));
      CHECK(!grad || q.piece <= (INT64_C(1) << 21));
      CHECK(q.total == need);
      const int64_t last_size = grad ? (int64_t)q.acc_tiles * (h.tokens <= 64 ? 64 : 256) * 1024
                                     : q.rows * 4;
      CHECK((grad ? q.o_acc : q.o_entry) + last_size <= q.total);
      if (grad) {
        CHECK(q.o_g + (size_t)(q.planes * q.rows * q.piece * 2) <= q.o_acc);
        CHECK((q.rows / (h.tokens <= 64 ? 256 : 256)) * ((q.dimp + 255) / 256) <= q.acc_tiles);
      } else {
        CHECK(q.stat_cols * 128 >= h.vocab);
        CHECK(q.o_stat + (size_t)(q.rows * q.stat_cols * 8) <= q.o_sum);
      }
      if (q.pack_w)
        CHECK(q.o_w + (size_t)(q.planes * q.piece * q.dimp * 2) <= (grad ? q.o_rowp : q.o_stat));
    }
  }
  CHECK(zero_loss_workspace_bytes(nullptr, 0, nullptr) == ZERO_EINVAL);
  std::printf("loss host layer: %d failures\n", failures);
  return failures != 0;
}
