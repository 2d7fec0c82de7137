// Prints what the library plans for a cache call: B H H_kv d block max_blocks rows max_new weights, read from the
// arguments -> workers, whole_row_tiles, wide_join, join_ctas, line_places. Host code only.
#include <cstdio>
#include <cstdlib>

#include "serving.h"

int main(int argc, char** argv) {
  if (argc != 10) return 1;
  auto arg = [&](int i) { return atoi(argv[i]); };
  sda::Cache c{};
  c.B = arg(1);
  c.H = arg(2);
  c.H_kv = arg(3);
  c.g = c.H / c.H_kv;
  c.d = arg(4);
  c.block = arg(5);
  c.n_blocks = 1;
  c.max_blocks = arg(6);
  c.rows = arg(7);
  c.max_new = arg(8);
  c.weights = arg(9);
  const sda::CacheLayout y = sda::make_cache_layout(c);
  printf("%d %d %d %lld %lld\n", y.workers, y.whole_row_tiles, y.wide_join, y.join_ctas, y.line_places);
  return 0;
}
