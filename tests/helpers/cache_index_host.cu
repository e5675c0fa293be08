// The cache's index arithmetic, run on the CPU: reads lines "name args..." from
// stdin, writes one result per line. No device code is involved.
#include <cstdio>
#include <cstring>

#include "../../quantized_attention_fp64_gb300/csrc/cache.cuh"

int main() {
  char name[32];
  while (std::scanf("%31s", name) == 1) {
    long long a, b, c, d, e;
    if (!std::strcmp(name, "capacity") && std::scanf("%lld %lld", &a, &b) == 2) {
      std::printf("%lld\n", static_cast<long long>(sage::table_capacity(a, static_cast<int32_t>(b))));
    } else if (!std::strcmp(name, "length") && std::scanf("%lld %lld", &a, &b) == 2) {
      bool bad = false;
      const long long r = sage::checked_length(a, b, &bad);
      std::printf("%lld %d\n", r, bad ? 1 : 0);
    } else if (!std::strcmp(name, "page") && std::scanf("%lld %lld", &a, &b) == 2) {
      std::printf("%d\n", sage::page_ok(a, b) ? 1 : 0);
    } else if (!std::strcmp(name, "slot") && std::scanf("%lld %lld %lld %lld %lld", &a, &b, &c, &d, &e) == 5) {
      std::printf("%lld\n", static_cast<long long>(sage::block_slot(a, static_cast<int32_t>(b), static_cast<int32_t>(c),
                                                                    static_cast<int32_t>(d), static_cast<int32_t>(e))));
    } else if (!std::strcmp(name, "position") && std::scanf("%lld", &a) == 1) {
      const int p = sage::value_position(static_cast<int>(a));
      std::printf("%d %d\n", p, sage::value_token(p));
    } else {
      return 1;
    }
  }
  return 0;
}
