// The checks of kv_plan_check.cpp on the shapes that the kernels use: their row
// tiles, units and item weights, on the grids of a device of 152 SMs; and the
// parts of one sequence of 4097 keys that the few-row kernel's comment states.
#define main base_main
#include "kv_plan_check.cpp"
#undef main

int main() {
  if (base_main()) return 1;
  struct { int RT, per, extra, grid; } variants[] = {
      {8, 8, 6, 304}, {16, 8, 6, 304}, {8, 16, 6, 304}, {16, 16, 6, 304},   // few rows: 96 and 128 wide, 64 wide
      {256, 4, 10, 152}, {128, 4, 4, 152}, {128, 4, 8, 152}};              // many rows: bf16, two parts, 64 wide
  unsigned rng = 777;
  const auto next = [&](int m) {
    rng = rng * 1664525u + 1013904223u;
    return (int)(rng >> 8) % m;
  };
  int n = 0;
  for (const auto& v : variants)
    for (int round = 0; round < 40; ++round) {
      const KvShape c{1 + next(8), v.RT, v.per, v.extra, next(2), next(3) ? 0 : 1 + next(300)};
      std::vector<Seq> seqs;
      const int batch = 1 + next(round % 5 ? 6 : 60), big = round % 7 ? 300 : 5000;
      for (int i = 0; i < batch; ++i)
        seqs.push_back(Seq{next(4) ? (v.RT < 100 ? next(6) : next(400)) : next(2), next(5) ? next(big) : next(3)});
      if (check(c, seqs, 1 + next(8), v.grid)) {
        std::printf("RT %d per %d extra %d, round %d\n", v.RT, v.per, v.extra, round);
        return 1;
      }
      ++n;
    }
  // one token on 4097 keys, 8 heads of 128 with 4 query heads each: 33 units a head of weight 39
  const KvShape c{4, 8, 8, 6, 1, 0};
  const long long head = kv_head_weight(c, 1, 4097), U = 8 * head;
  CHECK(head == 39);
  int most = 0;
  for (int h = 0; h < 8; ++h) {
    const long long first = h * head + c.extra;
    const int parts = kv_owner(first + 32, U, 304) - kv_owner(first, U, 304) + 1;
    if (parts > most) most = parts;
  }
  CHECK(most == 32);
  std::printf("ok %d batches of the variants, %d parts\n", n, most);
  return 0;
}
