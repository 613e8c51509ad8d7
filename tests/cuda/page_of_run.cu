// The append's page lookup on the host: lines "first len nth" in, "first p0 from to page" out.
#include <cstdio>

#include "../../quantized_kv_cache_kvq_gb300/csrc/runs.cuh"

int main() {
  int first, len, nth;
  while (std::scanf("%d %d %d", &first, &len, &nth) == 3) {
    const kvq::runs::RunPage p = kvq::runs::page_of_run(first, len, nth);
    std::printf("%d %d %d %d %d\n", p.first, p.p0, p.from, p.to, p.page);
  }
  return 0;
}
