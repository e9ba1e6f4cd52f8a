// kernels_attn.hip -- attention of drafted tokens over a paged cache
// (attn_kernels.hpp), and how its calls are cut.
#include "attn_kernels.hpp"

namespace lg {

namespace {

// What the rows of a tile of so many nodes count over with a window at most: sinks
// and window end in blocks of up to 128.
int64_t window_reach(int64_t window, int64_t sinks, int64_t nodes) { return sinks + window + nodes + 256; }

// The tile kernel with a window: how many positions a row tile goes over hardly
// depends on the context, so whole rounds of 256 workgroups count, and parts of
// splits, which go through memory, cost more than they do over long contexts.
// The form with the least of
//   rounds (start + per 128 positions) + (splits > 1: 4 + parts written and read)
// in us.  Measured with 32 query and 8 key heads of 128: 2 x 1500 nodes over 5001
// positions, window 1024: 256 rows whole 106 us, 128 rows 109 and in two splits 175;
// window 4096: 288 and 285; 8 trees of 64 nodes: 61, 42 and 43; 200 nodes: 49, 34
// and (128 rows in four splits) 28.  Dim 64, 2 x 1500 nodes: 85 and 82; dim 256,
// 2 x 700: 176 and (two splits) 212, with 8 query and 2 key heads 89 and 73.
AttnPlan window_plan(int64_t B, int Hk, int G, int D, int64_t max_nodes, int64_t max_len, int64_t all_rows,
                     int64_t window, int64_t sinks, bool masked) {
  AttnPlan best = {AT_TILE128, false, 1, 1, 128};
  double least = 0;
  const int64_t rows = max_nodes * G;
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 27) / (all_rows * (D + 2) * (int64_t)sizeof(float)));
  for (int shape : {AT_TILE128, AT_TILE256}) {
    if (shape == AT_TILE256 && (D == 256 || rows <= 32)) continue;
    const int bm = attn_rows(shape);
    // a tile holds bm / G nodes and parts of two more, or a whole tree
    const int64_t nodes = masked ? max_nodes : std::min<int64_t>(max_nodes, bm / G + 2);
    const int64_t len = std::min(max_len, window_reach(window, sinks, nodes));
    const int64_t tiles = (rows + bm - 1) / bm, units = B * Hk * tiles;
    const int64_t steps = (len + 127) / 128;  // whole blocks of any kernel
    const double start = D == 256 ? 23 : shape == AT_TILE256 ? 11 : 8;
    const double per = D == 256 ? 6.7 : shape == AT_TILE256 ? (D == 64 ? 2.7 : 3.75) : (D == 64 ? 1.85 : 2.5);
    for (int64_t n = 1; n <= std::min({(int64_t)16, steps, most}); ++n) {
      const int64_t each = (steps + n - 1) / n;
      if ((steps + each - 1) / each != n) continue;  // the same cut as with fewer
      double t = (double)((units * n + 255) / 256) * (start + per * (double)each);
      if (n > 1) t += 4 + (double)(n * all_rows * D) * 8 / 4.5e6;
      if (least > 0 && t >= least) continue;
      least = t;
      best = {shape, false, tiles, n, each * 128};
    }
  }
  return best;
}

}  // namespace

AttnPlan attn_plan(int64_t B, int Hk, int G, int D, int64_t max_nodes, int64_t max_len,
                   int64_t all_rows, int64_t window, int64_t sinks, bool masked) {
  AttnPlan p;
  const int64_t rows = max_nodes * G;
  if (window > 0) {
    if (rows > 16) return window_plan(B, Hk, G, D, max_nodes, max_len, all_rows, window, sinks, masked);
    max_len = std::min(max_len, window_reach(window, sinks, max_nodes));
  }
  // (Measured at dim 128 over 16-bit caches of thousands of positions; the other
  // dims, codes and short contexts follow the same borders unmeasured.)
  // 8 trees over 8000 positions (dim 128, bf16), rows of a key head: 32 rows
  // take 67 us in tiles of 128 and 83 in two tiles of the streaming kernel, 128
  // rows 82 and (tiles of 256) 88, 192 rows 118 and 101.  16 rows stream: 48
  // sequences of 8-bit codes take 127 us, and 231 in tiles of 128.
  if (D == 256) p.shape = rows <= 16 ? AT_STREAM16 : AT_TILE128;  // what fits the registers
  else p.shape = rows <= 16 ? AT_STREAM16 : rows <= 128 ? AT_TILE128 : AT_TILE256;
  const int bm = attn_rows(p.shape);
  p.ntiles = (rows + bm - 1) / bm;
  const int64_t units = B * Hk * p.ntiles;
  const int64_t step = p.shape == AT_STREAM16 ? 128 : 64;  // positions of one round of the waves
  const int64_t steps = (max_len + step - 1) / step;
  // Parts of splits take 128 MB at most, so that a call's workspace is bounded.
  // (With 32 heads of 128: 2100 nodes over 5000 positions take 390 us in nine
  // splits of 35 MB and 322 in three; 3 x 1400 over 2000 432 and 289; 4200 over
  // 12000 1254 in four of 70 MB, and 1353 whole.)
  const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 27) / (all_rows * (D + 2) * (int64_t)sizeof(float)));
  int64_t ns;
  if (p.shape == AT_STREAM16) {
    // A workgroup for each CU; more make more parts to join (one sequence of
    // 8000 positions: 14.8 us with 256, 17.9 with 512).  Lengths may differ,
    // though: up to 1536 where a split is longer than 2048 positions (48
    // sequences of up to 8191, 8-bit: 143 us with 768, 127 with 1536).
    ns = (256 + units - 1) / units;
    if (units * ns < 1536) ns = std::max(ns, std::min((1536 + units - 1) / units, (max_len + 2047) / 2048));
    ns = std::min({ns, steps, most});
  } else {
    // as many as fill whole rounds best; splits of four tiles at least
    const int64_t slots = 256;
    double best = 0;
    ns = 1;
    for (int64_t n = 1; n <= std::min({(int64_t)16, (steps + 3) / 4, most}); ++n) {
      const int64_t rounds = (units * n + slots - 1) / slots;
      const double use = (double)(units * n) / (double)(rounds * slots) - 0.01 * (double)n;
      if (use > best + 1e-9) { best = use; ns = n; }
    }
  }
  ns = std::max<int64_t>(1, ns);
  p.chunk = (steps + ns - 1) / ns * step;
  p.nsplit = std::max<int64_t>(1, (max_len + p.chunk - 1) / p.chunk);
  // Joined by the last workgroup, a call of one token over 1024 positions
  // takes 10.3 instead of 12 us; of 1536 workgroups (48 sequences of up to 8191)
  // the arrivals and the narrower stores cost 5 us more than a second launch.
  p.arrival = p.shape == AT_STREAM16 && units * p.nsplit <= 512;
  return p;
}

hipError_t launch_attention(const AttnArgs& a, int D, int shape, bool f16, bool kv8, hipStream_t s) {
  return launch_any(a, D, shape, f16, kv8, s);
}

}  // namespace lg
