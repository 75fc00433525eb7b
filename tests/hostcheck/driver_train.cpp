// Sanitizer driver for the host side of the training operators (tests/test_train_host.py builds it with
// -fsanitize=address,undefined and runs it on the CPU): the entry points over a sweep of sizes with each
// launch's buffers and workspace regions checked (stubs_train.cpp); the deals of tiles to workgroups,
// which the kernels share, against a list of what has to be done; the bounds of the launches. "Device"
// buffers are reserved address ranges that nothing reads.
#include <sys/mman.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../../include/beam_moe.h"
#include "../../routing_grouped_expert_fp32_amd/csrc/train_rules.h"
#include "hostcheck_train.h"

void* hostcheck::scratch_range() { return nullptr; }   // no entry point here takes it

namespace {

using beam::ceil_div;

long g_checks = 0;
int g_fail = 0;

void expect(bool ok, const char* what, long a = 0, long b = 0, long c = 0, long d = 0) {
  ++g_checks;
  if (!ok && ++g_fail <= 20)
    std::fprintf(stderr, "FAIL: %s (%ld, %ld, %ld, %ld)\n", what, a, b, c, d);
}

std::vector<std::pair<void*, size_t>> g_maps;
// A reserved, never-touched address range of `bytes` (page-aligned), registered for the stubs.
void* buf(size_t bytes, const char* name) {
  const size_t n = bytes ? (bytes + 4095) & ~size_t(4095) : 4096;
  void* p = mmap(nullptr, n, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
  if (p == MAP_FAILED) {
    std::perror("mmap");
    std::exit(2);
  }
  hostcheck::register_range(p, bytes, name);
  g_maps.push_back({p, n});
  return p;
}
void release() {
  for (auto& m : g_maps) munmap(m.first, m.second);
  g_maps.clear();
  hostcheck::clear_ranges();
}

std::mt19937 g_rng(1);
int64_t spread(int64_t lo, int64_t hi) {
  return std::llround(std::exp(std::uniform_real_distribution<double>(
      std::log((double)lo), std::log((double)hi))(g_rng)));
}
int64_t pick(int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(g_rng); }

// ---- entry points ---------------------------------------------------------------------------------
void grouped_calls(int64_t R, int32_t E, int32_t N, int32_t K, int32_t dt) {
  const size_t r = R, e = E, n = N, k = K, ob = dt == BEAM_BF16 ? 2 : 4;
  void* x = buf(2 * r * k, "x");
  void* dy = buf(2 * r * n, "dy");
  void* w = buf(2 * e * n * k, "w");
  int32_t* off = (int32_t*)buf(4 * (e + 1), "offsets");
  const long l0 = hostcheck::train_launches();
  expect(beam_moe_grouped_mm(x, w, off, buf(ob * r * n, "y"), R, E, N, K, dt, nullptr) == BEAM_OK,
         "grouped_mm", R, E, N, K);
  expect(beam_moe_grouped_mm_dx(dy, w, off, buf(ob * r * k, "dx"), R, E, N, K, dt, nullptr) == BEAM_OK,
         "grouped_mm_dx", R, E, N, K);
  expect(beam_moe_grouped_mm_dw(dy, x, off, buf(ob * e * n * k, "dw"), R, E, N, K, dt, nullptr) ==
             BEAM_OK,
         "grouped_mm_dw", R, E, N, K);
  expect(hostcheck::train_launches() - l0 == (R ? 3 : 1), "launches", R, E, N, K);
  release();
}

void boundary_calls(int64_t T, int32_t H, int32_t dt) {
  const size_t th = (size_t)T * H, gb = 4 * (size_t)H, yb = dt == BEAM_BF16 ? 2 : 4;
  const size_t need = beam_residual_boundary_backward_workspace_bytes(T, H);
  void* y = buf(yb * th, "y");
  void* h = buf(2 * th, "h_out");
  float* gp = (float*)buf(gb, "gamma_post");
  float* gn = (float*)buf(gb, "gamma_next");
  void* dh = buf(2 * th, "d_h_out");
  void* dx = buf(2 * th, "d_x_next");
  void* d_y = buf(yb * th, "d_y");
  void* d_h = buf(2 * th, "d_h");
  float* dgp = (float*)buf(gb, "d_gamma_post");
  float* dgn = (float*)buf(gb, "d_gamma_next");
  void* ws = buf(need, "workspace");
  auto call = [&](const void* in, void* out, size_t bytes) {
    return beam_residual_boundary_backward(y, dt, h, gp, gn, in, dx, d_y, out, dgp, dgn, T, H, 7,
                                           1e-6f, ws, bytes, nullptr);
  };
  expect(call(dh, d_h, need) == BEAM_OK, "boundary backward", T, H);
  expect(call(dh, dh, need) == BEAM_OK, "boundary backward in place", T, H);
  expect(call(nullptr, d_h, need) == BEAM_OK, "boundary backward without d_h_out", T, H);
  if (T > 0) expect(call(dh, d_h, need - 1) == BEAM_ERR_WORKSPACE, "boundary workspace", T, H);
  if (T > 0) expect(call(dh, (char*)dh + 16, need) == BEAM_ERR_ALIAS, "boundary alias", T, H);
  release();
}

void orthogonalise_calls(int64_t n, int32_t rows, int32_t cols, int32_t dt) {
  const float abc[3] = {3.4445f, -4.775f, 2.0315f};
  const size_t count = (size_t)n * rows * cols;
  const size_t need = beam_moe_orthogonalise_workspace_bytes(n, rows, cols);
  expect(need > 0 && need == beam_moe_orthogonalise_workspace_bytes(n, cols, rows), "workspace", n, rows,
         cols);
  void* g = buf((dt == BEAM_BF16 ? 2 : 4) * count, "g");
  void* out = buf(2 * count, "out");
  void* ws = buf(need, "workspace");
  for (int steps : {1, 5, 64})
    expect(beam_moe_orthogonalise(g, dt, out, n, rows, cols, steps, abc, 1e-7f, ws, need, nullptr) ==
               BEAM_OK,
           "orthogonalise", n, rows, cols, steps);
  expect(beam_moe_orthogonalise(g, dt, out, n, rows, cols, 5, abc, 1e-7f, ws, need - 1, nullptr) ==
             BEAM_ERR_WORKSPACE,
         "orthogonalise workspace", n, rows, cols);
  release();
}

// ---- deals ----------------------------------------------------------------------------------------
constexpr int64_t kMaxThreads = int64_t(1) << 32;

// Rows of E experts, some without, some with most.
std::vector<int> random_counts(int64_t R, int E) {
  std::vector<int> c(E, 0);
  const int hot = (int)pick(0, E - 1), kind = (int)pick(0, 2);
  int64_t left = R;
  if (kind == 1) {
    c[hot] = (int)(R / 2);
    left -= c[hot];
  } else if (kind == 2) {
    c[hot] = (int)R;
    left = 0;
  }
  for (int64_t i = 0; i < 4 * E && left > 0; ++i) {
    const int64_t n = std::min(left, pick(0, 2 * R / E + 1));
    c[pick(0, E - 1)] += (int)n;
    left -= n;
  }
  return c;   // the rest belongs to no expert
}

// Forward and input gradient: every column tile of every block of rows is some workgroup's, once.
void rows_deal(int64_t R, int E, int No, int Kc, bool bf16) {
  const std::vector<int> counts = random_counts(R, E);
  beam::with_rows_tile(R, E, No, Kc, bf16, [&](auto s) {
    using S = decltype(s);
    const int64_t blocks = beam::grouped_max_blocks(R, E, S::BM);
    const int n_ctiles = (int)ceil_div(No, S::BN);
    const int64_t wgs = beam::xcd_workgroups_halves<S>(blocks * n_ctiles);
    expect(wgs * S::kThreads < kMaxThreads, "threads", R, E, No, Kc);
    std::vector<int> expert, in_expert;   // of a block
    for (int e = 0; e < E; ++e) {
      const int n = beam::blocks_of<S::BM>(counts[e]);
      int next = 0;
      for (int i = 0; i < n; ++i) {
        expert.push_back(e);
        in_expert.push_back(i);
        int first = -1, rows = -1;
        beam::block_rows<S::BM>(counts[e], n, i, first, rows);
        expect(first == next && rows > 0 && rows <= S::BM, "block's rows", counts[e], n, i, S::BM);
        next = first + rows;
      }
      expect(next == counts[e], "blocks hold an expert's rows", counts[e], n, S::BM);
    }
    expect((int64_t)expert.size() <= blocks, "bound on the blocks", R, E, (long)expert.size());
    const int total = (int)expert.size() * n_ctiles;
    std::vector<unsigned char> seen((size_t)total, 0);   // 1, 2: halves, 3: whole
    std::vector<int> first_block(E, 0);
    for (int b = (int)expert.size() - 1; b >= 0; --b) first_block[expert[b]] = b;
    for (int64_t wg = 0; wg < wgs; ++wg) {
      int half = -1;
      const int v = beam::xcd_tile_halves<S>((int)wg, total, half);
      if (v < 0) continue;
      if (v >= total) {
        expect(false, "tile in range", R, E, v);
        return;
      }
      const int b = v / n_ctiles, e = expert[b], n = beam::blocks_of<S::BM>(counts[e]);
      int block = -1, ctile = -1;
      beam::group_tile(v, b, in_expert[b], n, n_ctiles, block, ctile);
      if (block < 0 || block >= n || ctile < 0 || ctile >= n_ctiles) {
        expect(false, "block and column tile in range", v, block, ctile);
        return;
      }
      unsigned char& f = seen[(size_t)(first_block[e] + block) * n_ctiles + ctile];
      const unsigned char bit = half < 0 ? 3 : (unsigned char)(1 << half);
      expect((f & bit) == 0, "tile dealt once", v, block, ctile, half);
      f |= bit;
    }
    bool all = true;
    for (unsigned char f : seen) all = all && f == 3;
    expect(all, "every tile dealt", R, E, No, Kc);
  });
}

// Weight gradient: every tile of every expert's matrix, once.
void dw_deal(int64_t R, int E, int N, int K, bool bf16) {
  beam::with_dw_tile(R, E, N, K, bf16, [&](auto s) {
    using S = decltype(s);
    const int n_mtiles = (int)ceil_div(N, S::BM), n_ctiles = (int)ceil_div(K, S::BN);
    const int per = n_mtiles * n_ctiles;
    const int64_t wgs = beam::dw_workgroups(per, E);
    expect(wgs * S::kThreads < kMaxThreads, "threads", R, E, N, K);
    std::vector<unsigned char> seen((size_t)per * E, 0);
    for (int64_t wg = 0; wg < wgs; ++wg) {
      int pos = -1, t = -1, mt = -1, ct = -1;
      if (!beam::dw_tile((unsigned)wg, per, E, pos, t)) continue;
      beam::band_tile(t, n_mtiles, n_ctiles, mt, ct);
      const bool in = pos >= 0 && pos < E && mt >= 0 && mt < n_mtiles && ct >= 0 && ct < n_ctiles;
      expect(in && !seen[((size_t)pos * n_mtiles + mt) * n_ctiles + ct], "tile dealt once", E, N, K, wg);
      if (!in) return;
      seen[((size_t)pos * n_mtiles + mt) * n_ctiles + ct] = 1;
    }
    bool all = true;
    for (unsigned char f : seen) all = all && f;
    expect(all, "every tile dealt", E, N, K);
  });
}

// Any count of tiles, with and without halves.
template <class S>
void xcd_deal(int total, int64_t bound) {
  std::vector<unsigned char> seen((size_t)total, 0), plain((size_t)total, 0);
  for (int64_t wg = 0; wg < beam::xcd_workgroups_halves<S>(bound); ++wg) {
    int half = -1;
    const int v = beam::xcd_tile_halves<S>((int)wg, total, half);
    if (v >= 0 && v < total) seen[v] += half < 0 ? 3 : 1 << half;
    expect(v < total, "tile in range", total, v);
  }
  for (int64_t wg = 0; wg < beam::xcd_workgroups(bound); ++wg) {
    const int v = beam::xcd_tile((int)wg, total);
    if (v >= 0 && v < total) plain[v] += 1;
    expect(v < total, "tile in range", total, v);
  }
  bool all = true;
  for (int i = 0; i < total; ++i) all = all && seen[i] == 3 && plain[i] == 1;
  expect(all, "every tile once", total, (long)bound);
}

// ---- bounds of the launches at the limits of the sizes -----------------------------------------------
void limits() {
  long fit = 0;
  for (int i = 0; i < 20000; ++i) {
    const int64_t R = spread(1, (int64_t(1) << 31) - 1), E = spread(1, 4096);
    const int64_t N = 8 * spread(1, 1 << 17), K = 8 * spread(1, 1 << 17);
    if (N * K >= (int64_t(1) << 31) || !beam::grouped_grid_fits(R, E, N, K)) continue;
    ++fit;
    for (bool bf16 : {false, true}) {
      for (bool across : {false, true}) {
        const int64_t No = across ? K : N, Kc = across ? N : K;
        beam::with_rows_tile(R, E, No, Kc, bf16, [&](auto s) {
          using S = decltype(s);
          const int64_t tiles = beam::grouped_max_blocks(R, E, S::BM) * ceil_div(No, S::BN);
          expect(beam::xcd_workgroups_halves<S>(tiles) * S::kThreads < kMaxThreads &&
                     tiles < (int64_t(1) << 31),
                 "rows' launch", R, E, No, Kc);
        });
      }
      beam::with_dw_tile(R, E, N, K, bf16, [&](auto s) {
        using S = decltype(s);
        expect(beam::dw_workgroups(ceil_div(N, S::BM) * ceil_div(K, S::BN), E) * S::kThreads <
                   kMaxThreads,
               "weight gradient's launch", R, E, N, K);
      });
    }
  }
  expect(fit > 5000, "sizes that fit", fit);
  fit = 0;
  for (int i = 0; i < 20000; ++i) {
    const int64_t n = spread(1, 65535);
    const int rows = (int)spread(1, 1 << 16), cols = (int)spread(1, 1 << 16);
    if (!beam::ns_grid_fits(n, rows, cols)) continue;
    ++fit;
    const beam::NsLayout L = beam::ns_layout(n, rows, cols);
    if (beam::ns_is_small(L.m, L.n)) {
      expect(n * 512 < kMaxThreads, "one launch", n, rows, cols);
      continue;
    }
    auto gram = [&](int side) { return n * beam::ns_triangle(ceil_div(L.m, side)); };
    auto update = [&](int side) { return n * ceil_div(L.m, side) * ceil_div(L.ld, side); };
    auto fits = [&](const char* what, int64_t wgs, int threads) {
      expect(wgs < (int64_t(1) << 31) && wgs * threads < kMaxThreads, what, n, rows, cols);
    };
    beam::with_ns_tile(false, L.n, gram, [&](auto t) {
      using S = decltype(t);
      fits("A's launch", beam::xcd_workgroups(gram(S::BM)), S::kThreads);
    });
    beam::with_ns_tile(false, L.m, gram, [&](auto t) {
      using S = decltype(t);
      fits("B's launch", beam::xcd_workgroups(gram(S::BM)), S::kThreads);
    });
    beam::with_ns_tile(true, L.m, update, [&](auto t) {
      using S = decltype(t);
      fits("update's launch", beam::xcd_workgroups_halves<S>(update(S::BM)), S::kThreads);
    });
    const beam::GramParts split = beam::gram_parts(n, L.m, L.n);
    if (split.parts > 1) {
      fits("parts' launch", gram(64) * split.parts, beam::NsTile64::kThreads);
      fits("sums' launch", gram(64) * 4, 256);
    }
    fits("init's launch", ceil_div(L.ld, 64) * ceil_div(L.m, 64) * n, 256);
    fits("norm's launch", n * beam::ns_norm_parts((int64_t)rows * cols), 256);
  }
  expect(fit > 5000, "sizes that fit", fit);
}

}  // namespace

int main() {
  const int32_t types[] = {BEAM_F32, BEAM_BF16};
  for (int64_t R : {0, 1, 2, 63, 64, 65, 1000, 8192, 32768})
    for (int32_t E : {1, 3, 32, 256}) {
      grouped_calls(R, E, 5120, 2560, BEAM_BF16);
      grouped_calls(R, E, 8, 8, BEAM_F32);
    }
  for (int i = 0; i < 200; ++i)
    grouped_calls(spread(1, 1 << 20), (int32_t)spread(1, 4096), 8 * (int32_t)spread(1, 512),
                  8 * (int32_t)spread(1, 512), types[i & 1]);
  for (int64_t T : {0, 1, 2, 255, 256, 257, 511, 512, 513, 8192, 1 << 20})
    for (int32_t H = 256; H <= 16384; H += T == 513 ? 256 : 2560)
      for (int32_t dt : types) boundary_calls(T, H, dt);
  for (int32_t rows : {1, 7, 63, 64, 65, 127, 128, 129, 256, 2000})
    for (int32_t cols : {1, 8, 65, 383, 385, 1024, 1025, 5120})
      for (int64_t n : {1, 2, 26}) orthogonalise_calls(n, rows, cols, types[n & 1]);
  for (int i = 0; i < 300; ++i)
    orthogonalise_calls(spread(1, 40), (int32_t)spread(1, 9000), (int32_t)spread(1, 9000), types[i & 1]);
  expect(beam_moe_orthogonalise_workspace_bytes(1, 65536, 65536) > 0, "largest matrix");

  for (int i = 0; i < 600; ++i) {
    const int64_t R = spread(1, 40000);
    const int E = (int)spread(1, 300), N = 8 * (int)spread(1, 700), K = 8 * (int)spread(1, 700);
    rows_deal(R, E, N, K, i & 1);
    if (i % 4 == 0) dw_deal(R, 1 + E / 4, N, K, i & 1);
  }
  for (int total = 1; total < 1200; ++total) {
    xcd_deal<beam::Tile320>(total, total + total % 5 * 40);
    if (total % 7 == 0) xcd_deal<beam::TilePair>(total, total);
  }
  limits();
  std::printf("hostcheck: %ld checks, %d failed, %ld launches checked\n", g_checks, g_fail,
              hostcheck::train_launches());
  return g_fail ? 1 : 0;
}
