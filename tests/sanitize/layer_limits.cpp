// layer_limits.cpp - the layer entry points' host plans at the limits of rows
// and blocks of rows, and the areas that only some calls have.
// tests/test_layer_limits.py builds it with the library's host-only sources
// under the address and undefined-behaviour sanitizers.
#include <cstdint>
#include <cstdio>
#include <random>

#include "sgmv.h"
#include "sgmv_layer_host.h"

using namespace sgmv_host;

static int failures = 0;
#define CHECK(c)                                                          \
  do {                                                                    \
    if (!(c)) {                                                           \
      if (failures < 20) std::fprintf(stderr, "FAIL %s:%d: %s\n", __FILE__, __LINE__, #c); \
      ++failures;                                                         \
    }                                                                     \
  } while (0)

int main() {
  std::mt19937_64 rng(11);
  int taken = 0, refused = 0;
  for (int trial = 0; trial < 60000; ++trial) {
    sgmv_problem_t p{};
    p.dtype = (int32_t)(rng() % 2);
    p.n_rows = (int32_t)((rng() % (((uint64_t)1 << 31) - 1)) >> (rng() % 31));
    p.h_in = (int32_t)(1 + (rng() % (1 << 17) >> (rng() % 17))) * 8;
    p.h_out = (int32_t)(1 + (rng() % (1 << 17) >> (rng() % 17))) * 8;
    if (p.n_rows > 1 << 20) p.h_in = 8, p.h_out = 16;
    p.rank = 8 << (rng() % 4);
    p.num_loras = (int32_t)(1 + (rng() % (1 << 20) >> (rng() % 20)));
    p.num_segs = (int32_t)((rng() % (((uint64_t)1 << 31) - 1)) >> (rng() % 31));
    p.max_seg_len = p.n_rows ? (int32_t)(1 + (rng() % p.n_rows >> (rng() % 31))) : 0;
    p.variant = (int32_t)(rng() % 9);
    p.splits = (int32_t)rng();
    if (p.max_seg_len > p.n_rows) p.max_seg_len = p.n_rows;
    for (int op = 0; op < 4; ++op) {
      size_t bytes = 0;
      const sgmv_status_t st = sgmv_layer_workspace_bytes(&p, op, &bytes);
      int direct = 0;
      const bool fits = p.n_rows <= SGMV_MAX_LAYER_ROWS &&
                        (nothing_to_do(p) || (units_for(p, sgmv::kThinRows, &direct) <= SGMV_MAX_LAYER_UNITS &&
                                              (direct || p.num_segs <= SGMV_MAX_LAYER_LONG_SEGS)));
      CHECK(st == (fits ? SGMV_OK : SGMV_ERR_UNSUPPORTED));
      ++(fits ? taken : refused);
      if (st != SGMV_OK) continue;
      const LayerPlan l = plan_layer(p, op);
      CHECK(bytes == l.total);
      if (l.lora) {
        for (const ThinPlan* t : {&l.down, &l.up}) {  // one launch: fewer than 2^32 threads
          if (t == &l.up && !layer_backward(op)) continue;
          CHECK(t->units >= 1 && (int64_t)t->units * t->ksplit * 256 < (int64_t)1 << 32);
        }
      }
      CHECK(l.row_powers == (op == SGMV_GATED_BACKWARD && p.dtype == SGMV_F16));
      if (l.row_powers && p.n_rows > 0) {
        // Behind dG and dU, before the planes; readable to the next 32 rows.
        CHECK(l.row_power_off % 256 == 0);
        CHECK(l.row_power_off >= l.gate_off[1] + (size_t)p.n_rows * l.halves * p.h_out * 2);
        CHECK(l.row_power_off + (size_t)round_up(p.n_rows, 32) <= l.planes_off);
      }
      if (l.one_launch) CHECK(l.row_k_off + (size_t)p.n_rows * l.projections * 4 <= l.planes_off);
    }
  }
  CHECK(taken > 1000 && refused > 1000);
  if (failures) return 1;
  std::puts("layer limits ok");
  return 0;
}
