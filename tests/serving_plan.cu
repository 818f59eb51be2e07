// Prints what the host plans of a decoding step over a cache, for tests/test_serving_plan.py:
//   instances   for every kernel of the own rows: kind D rows CTAs-an-SM planned-CTAs-an-SM
//   rows N      the rows of a CTA for 1 .. N query rows a key head
//   plan B H Hk nq np max_len D elem_bytes   prefix: split pairs steps units CTAs steps-a-CTA; SMs of the own rows
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "fa_serve_own.cuh"

namespace fa {
template <int Kind, int D, int R>
void instance() {
  using C = OwnCfg<Kind, D, R>;
  std::printf("%d %d %d %d %d\n", Kind, D, R, C::kPerSm, own_per_sm(R, C::kElem, D));
}
template <int Kind, int D>
void rows_of() {
  instance<Kind, D, 4>();
  instance<Kind, D, 8>();
  instance<Kind, D, 16>();
  instance<Kind, D, 24>();
}
template <int Kind>
void widths() {
  rows_of<Kind, 64>();
  rows_of<Kind, 128>();
}
}  // namespace fa

int main(int argc, char** argv) {
  if (argc > 1 && !std::strcmp(argv[1], "instances")) {
    fa::widths<fa::kE4m3>();
    fa::widths<fa::kBf16>();
    fa::widths<fa::kF16>();
  } else if (argc > 2 && !std::strcmp(argv[1], "rows")) {
    for (int r = 1; r <= std::atoi(argv[2]); ++r) std::printf("%d\n", fa::own_rows(r));
  } else if (argc > 9 && !std::strcmp(argv[1], "plan")) {
    int v[8];
    for (int i = 0; i < 8; ++i) v[i] = std::atoi(argv[2 + i]);
    const fa::ServePlan s = fa::serve_plan(v[0], v[2], v[1] / v[2] * v[3], v[4], v[5], v[6], v[7]);
    std::printf("%d %d %d %d %d %lld %d\n", s.pre.split, s.pre.pairs, s.pre.steps, s.pre.units, s.pre.ctas,
                s.pre.per_cta, s.own_sms);
  } else {
    return 1;
  }
  return 0;
}
