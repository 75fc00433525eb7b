// Sanitizer driver for the host side of the operators that close a training step (tests/test_step_host.py
// builds it with -fsanitize=address,undefined and runs it on the CPU): the entry points over a sweep of
// sizes with each launch's buffers and workspace regions checked (stubs_step.cpp), the plan of dx, the
// bounds of the launches. "Device" buffers are reserved address ranges that nothing reads.
#include <sys/mman.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../../include/beam_moe.h"
#include "../../routing_grouped_expert_fp32_amd/csrc/step_rules.h"
#include "hostcheck_step.h"

void* hostcheck::scratch_range() { return nullptr; }   // no entry point here takes it

namespace {

using beam::ceil_div;

long g_checks = 0;
int g_fail = 0;

void expect(bool ok, const char* what, long a = 0, long b = 0, long c = 0, long d = 0) {
  ++g_checks;
  if (!ok && ++g_fail <= 20) std::fprintf(stderr, "FAIL: %s (%ld, %ld, %ld, %ld)\n", what, a, b, c, d);
}

std::vector<std::pair<void*, size_t>> g_maps;
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

std::mt19937 g_rng(2);
int64_t spread(int64_t lo, int64_t hi) {
  return std::llround(std::exp(std::uniform_real_distribution<double>(std::log((double)lo), std::log((double)hi))(g_rng)));
}
int64_t pick(int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(g_rng); }

void gated_calls(int64_t R, int32_t E, int32_t F, int32_t K) {
  const size_t r = R, e = E, f = F, k = K;
  void* x = buf(2 * r * k, "x");
  void* w = buf(4 * e * f * k, "w");
  int32_t* off = (int32_t*)buf(4 * (e + 1), "offsets");
  void* gu = buf(4 * r * f, "gu");
  void* h = buf(2 * r * f, "h");
  const bool fits = 2 * (int64_t)F * K < (int64_t(1) << 30);
  const beam_status_t want = fits ? BEAM_OK : BEAM_ERR_UNSUPPORTED;
  for (int32_t round : {0, 1}) {
    expect(beam_moe_gated_mm(x, w, off, h, gu, R, E, F, K, round, nullptr) == want, "gated_mm", R, E, F, K);
    expect(beam_moe_gated_mm(x, w, off, h, nullptr, R, E, F, K, round, nullptr) == want, "gated_mm", R, E, F, K);
  }
  void* wd = buf(2 * e * f * k, "w_down");
  void* d_gu = buf(4 * r * f, "d_gu");
  float* s = (float*)buf(4 * r, "row_scale");
  float* ds = (float*)buf(4 * r, "d_row_scale");
  const size_t need = beam_moe_gated_mm_backward_workspace_bytes(R, F);
  void* ws = buf(need, "workspace");
  if (fits) {
    expect(beam_moe_gated_mm_backward(x, wd, gu, off, s, d_gu, h, ds, R, E, F, K, ws, need, nullptr) == BEAM_OK,
           "gated_mm_backward", R, E, F, K);
    expect(beam_moe_gated_mm_backward(x, wd, gu, off, nullptr, d_gu, h, nullptr, R, E, F, K, nullptr, 0, nullptr) ==
               BEAM_OK,
           "gated_mm_backward without scales", R, E, F, K);
    if (R > 0)
      expect(beam_moe_gated_mm_backward(x, wd, gu, off, s, d_gu, h, ds, R, E, F, K, ws, need - 1, nullptr) ==
                 BEAM_ERR_WORKSPACE,
             "gated workspace", R, E, F, K);
  }
  release();
}

void head_calls(int64_t T, int64_t V, int32_t H, int32_t dt) {
  const size_t t = T, v = V, h = H;
  void* x = buf(2 * t * h, "x");
  void* w = buf(2 * v * h, "w");
  int32_t* y = (int32_t*)buf(4 * t, "targets");
  float* loss = (float*)buf(4 * t, "loss");
  float* lse = (float*)buf(4 * t, "lse");
  float* d = (float*)buf(4 * t, "d_loss");
  void* dx = buf(2 * t * h, "dx");
  void* dw = buf((dt == BEAM_BF16 ? 2 : 4) * v * h, "dw");
  const size_t n1 = beam_head_loss_workspace_bytes(T, V, H), n2 = beam_head_loss_backward_workspace_bytes(T, V, H);
  void* w1 = buf(n1, "workspace");
  void* w2 = buf(n2, "workspace");
  for (float cap : {0.f, 30.f}) {
    expect(beam_head_loss(x, w, y, loss, lse, T, V, H, cap, w1, n1, nullptr) == BEAM_OK, "head_loss", T, V, H);
    expect(beam_head_loss_backward(x, w, y, lse, d, dx, dw, dt, T, V, H, cap, w2, n2, nullptr) == BEAM_OK,
           "head_loss_backward", T, V, H);
  }
  if (T > 0) {
    expect(beam_head_loss(x, w, y, loss, lse, T, V, H, 0.f, w1, n1 - 1, nullptr) == BEAM_ERR_WORKSPACE, "workspace", T, V, H);
    expect(beam_head_loss_backward(x, w, y, lse, d, dx, dw, dt, T, V, H, 0.f, w2, n2 - 1, nullptr) == BEAM_ERR_WORKSPACE,
           "workspace", T, V, H);
    const beam::HeadBwdLayout L = beam::head_bwd_layout(T, V, H);
    expect(L.cols * L.pieces >= V && L.cols * (L.pieces - 1) < V && L.pitch % 64 == 0 && L.pitch >= L.cols &&
               (L.pieces == 1 || L.cols % 256 == 0),
           "pieces", T, V, H, L.pieces);
    const int64_t dz = 2 * T * L.pitch, slack = 2 * T * 256;   // columns go by 256
    expect(dz <= beam::kHeadPieceBytes + slack || (L.cols <= beam::kHeadPieceCols && dz <= beam::kHeadMostBytes + slack) ||
               L.cols <= beam::kHeadLeastCols,
           "a piece's size", T, V, H, L.cols);
    expect(L.dx.kp % 64 == 0 && L.dx.kp * L.dx.parts >= L.cols && L.dx.kp * (L.dx.parts - 1) < L.cols, "parts", T, V, H,
           L.dx.parts);
    const int64_t bm = L.dx.side, bn = L.dx.side == 32 ? 128 : L.dx.side;
    expect(ceil_div(T, bm) * ceil_div(H, bn) * L.dx.parts * 512 < (int64_t(1) << 32), "threads of dx", T, V, H);
  }
  release();
}

void adamw_calls(int n, int32_t p, int32_t g, int32_t s, bool copy) {
  std::vector<beam_adamw_tensor> t(n);
  for (auto& a : t) {
    a.count = pick(0, 9) == 0 ? 0 : spread(1, 1 << 24);
    const size_t c = (size_t)a.count, sb = s == BEAM_F32 ? 4 : 1, blocks = 4 * ((c + 255) / 256);
    a.param = buf((p == BEAM_F32 ? 4 : 2) * c, "param");
    a.grad = buf((g == BEAM_F32 ? 4 : 2) * c, "grad");
    a.m = buf(sb * c, "m");
    a.v = buf(sb * c, "v");
    a.m_scale = s == BEAM_F32 ? nullptr : (float*)buf(blocks, "m_scale");
    a.v_scale = s == BEAM_F32 ? nullptr : (float*)buf(blocks, "v_scale");
    a.copy = copy ? buf(2 * c, "copy") : nullptr;
  }
  beam_adamw_cfg cfg = {};
  cfg.lr = 1e-3;
  cfg.beta1 = 0.9;
  cfg.beta2 = 0.95;
  cfg.eps = 1e-8;
  cfg.step = 4;
  std::vector<char> table(beam_moe_adamw_table_bytes(t.data(), n));
  auto check = [&]() { return beam_moe_adamw_table(t.data(), n, p, g, s, table.data(), table.size()); };
  expect(check() == BEAM_OK, "adamw_table", n);
  expect(n == 0 || beam_moe_adamw_table(t.data(), n, p, g, s, table.data(), table.size() - 1) == BEAM_ERR_WORKSPACE,
         "adamw_table bytes", n);
  // every chunk's entry, and the blocks before it
  int32_t used = 0;
  for (auto& a : t) used += a.count > 0;
  const size_t kHead = sizeof(beam::AdamwTableHead);
  int64_t chunk = 0, blocks = 0;
  int32_t k = 0;
  for (auto& a : t) {
    if (a.count == 0) continue;
    beam::AdamwEntry e;
    std::memcpy(&e, table.data() + kHead + k * sizeof(e), sizeof(e));
    expect(e.t.param == a.param && e.t.count == a.count && e.first == chunk && e.base256 == blocks, "an entry", n, k);
    for (int64_t c = 0; c < beam::adamw_chunks(a.count); ++c, ++chunk) {
      int32_t at;
      std::memcpy(&at, table.data() + kHead + used * sizeof(e) + 4 * chunk, 4);
      expect(at == k, "a chunk's entry", n, k, chunk);
    }
    blocks += ceil_div(a.count, 256);
    ++k;
  }
  if (n > 0) {
    beam::AdamwTableHead head;
    std::memcpy(&head, table.data(), sizeof(head));
    expect(head.entries == used && head.chunks == chunk && kHead + used * sizeof(beam::AdamwEntry) + 4 * chunk == table.size(),
           "the table's head", n);
  }
  void* on_device = buf(table.size(), "table");
  expect(beam_moe_adamw(t.data(), n, p, g, s, &cfg, nullptr, nullptr) == BEAM_OK, "adamw", n);
  expect(beam_moe_adamw(t.data(), n, p, g, s, &cfg, on_device, nullptr) == BEAM_OK, "adamw with its table", n);
  if (n > 1 && t[0].count > 300 && t[n - 1].count > 300) {   // arrays of two tensors that meet
    void* const was = t[0].m;
    t[0].m = (char*)t[n - 1].param + 16;
    expect(check() == BEAM_ERR_ALIAS, "adamw_check overlap", n);
    t[0].m = was;
    t[0].grad = t[n - 1].grad;   // gradients may
    if (t[0].count <= t[n - 1].count) expect(check() == BEAM_OK, "shared grads", n);
  }
  release();
}

// Every tile of a deal to one workgroup, whole or as its two halves.
template <class S>
void dealt(int total) {
  std::vector<int> whole(total, 0), halves(2 * total, 0);
  const int64_t wgs = beam::xcd_workgroups_halves<S>(total + pick(0, 40));   // a bound: the host knows no more
  for (int64_t wg = 0; wg < wgs; ++wg) {
    int half = 0;
    const int t = beam::xcd_tile_dealt<S>((int)wg, total, half);
    if (t < 0) continue;
    expect(t < total && half < 2 && (beam::kHalves<S> || half < 0), "a tile of the deal", total, wg, t, half);
    if (t >= total) continue;
    if (half < 0)
      ++whole[t];
    else
      ++halves[2 * t + half];
  }
  for (int t = 0; t < total; ++t)
    expect(whole[t] == 1 ? !halves[2 * t] && !halves[2 * t + 1] : !whole[t] && halves[2 * t] == 1 && halves[2 * t + 1] == 1,
           "dealt once", total, t, whole[t], halves[2 * t]);
}

// Launches of every accepted size stay under 2^32 threads.
void limits() {
  long fit = 0;
  for (int i = 0; i < 20000; ++i) {
    const int64_t R = spread(1, (int64_t(1) << 31) - 1), E = spread(1, 4096), F = 8 * spread(1, 1 << 16),
                  K = 8 * spread(1, 1 << 16);
    if (2 * F * K < (int64_t(1) << 30) && beam::gated_grid_fits(R, E, F, K)) {
      ++fit;
      for (bool keep : {false, true})
        beam::with_gated_tile(R, E, F, K, keep, [&](auto s) {
          using S = decltype(s);
          const int64_t tiles = beam::grouped_max_blocks(R, E, S::BM) * ceil_div(F, beam::kGatedCols<S>);
          expect(beam::xcd_workgroups_halves<S>(tiles) * S::kThreads < (int64_t(1) << 32) && tiles < (int64_t(1) << 31),
                 "gated threads", R, E, F, K);
        });
    }
    const int64_t T = spread(1, (int64_t(1) << 31) - 1), V = spread(1, 1 << 23), H = 8 * spread(1, 1 << 17);
    if (!beam::head_grid_fits(T, V, H)) continue;
    ++fit;
    expect(T * 256 < (int64_t(1) << 32) && ceil_div(T * H, 8 * 256) * 256 < (int64_t(1) << 32), "threads of rows", T, V, H);
    const beam::HeadBwdLayout L = beam::head_bwd_layout(T, V, H);
    const int64_t bm = L.dx.side, bn = L.dx.side == 32 ? 128 : L.dx.side;
    expect((ceil_div(T, bm) * ceil_div(H, bn) * L.dx.parts + 8) * 512 < (int64_t(1) << 32), "threads of dx", T, V, H);
    // what 32-bit offsets span: the rows of a tile of dz, 64 stored rows of dz, w and x
    expect(2 * std::min<int64_t>(T, 320) * L.pitch < (int64_t(1) << 31), "a tile's rows of dz", T, V, H);
    expect(2 * 64 * L.pitch < (int64_t(1) << 31) || T < 64, "a stage's rows of dz", T, V, H);
    for (bool store : {false, true})
      beam::with_head_tile(T, store ? L.cols : V, H, store, [&](auto s) {
        using S = decltype(s);
        const int64_t tiles = ceil_div(T, S::BM) * ceil_div(store ? L.pitch : V, S::BN);
        expect(beam::xcd_workgroups_halves<S>(tiles) * S::kThreads < (int64_t(1) << 32), "threads of logits", T, V, H);
      });
  }
  expect(fit > 5000, "sizes that fit", fit);
}

}  // namespace

int main() {
  for (int64_t R : {0, 1, 2, 63, 64, 65, 1000, 8192, 32768})
    for (int32_t E : {1, 3, 32, 256}) {
      gated_calls(R, E, 2560, 5120);
      gated_calls(R, E, 8, 8);
    }
  gated_calls(4096, 1, 20480, 5120);
  for (int i = 0; i < 200; ++i)
    gated_calls(spread(1, 1 << 20), (int32_t)spread(1, 4096), 8 * (int32_t)spread(1, 512), 8 * (int32_t)spread(1, 512));
  for (int64_t T : {0, 1, 2, 32, 203, 4096, 65536})
    for (int64_t V : {1, 63, 50003, 131072})
      for (int32_t H : {8, 1032, 5120}) head_calls(T, V, H, T & 1 ? BEAM_F32 : BEAM_BF16);
  for (int i = 0; i < 300; ++i)
    head_calls(spread(1, 1 << 18), spread(1, 1 << 20), 8 * (int32_t)spread(1, 1024), i & 1 ? BEAM_F32 : BEAM_BF16);
  for (int i = 0; i < 60; ++i)
    adamw_calls((int)spread(1, 200), i & 1 ? BEAM_F32 : BEAM_BF16, i & 2 ? BEAM_F32 : BEAM_BF16,
                i & 4 ? BEAM_F32 : BEAM_FP8_E4M3, (i & 1) && (i & 8));
  for (int total = 1; total < 1600; ++total) {
    dealt<beam::Tile320>(total);
    if (total % 7 == 0) dealt<beam::TilePair>(total);
  }
  limits();
  std::printf("hostcheck: %ld checks, %d failed, %ld launches checked\n", g_checks, g_fail, hostcheck::step_launches());
  return g_fail ? 1 : 0;
}
