// Host-side driver for test_host_attend_split.py: the split of units into runs, as the
// attention kernels and their joins form it, for every small size and many large ones.
// Runs have to follow one another without a gap, none may be empty, and the slot of a
// unit has to be the one whose run it lies in.  Exit status 0 when they do.
#include <stdio.h>

#include <random>

#include "../prng_seeded_decode_amd/csrc/attend_split.h"

namespace {

long g_bad = 0, g_runs = 0;

template <int GENS>
void check(int most, int units) {
  const seedlm::Runs<GENS> runs(most, units);
  bool good = runs.begin(0) == 0 && runs.begin(runs.slots) == units && runs.slots >= 1;
  int shortest = units, longest = 0;
  for (int s = 0; s < runs.slots; ++s) {
    const int b = runs.begin(s), e = runs.begin(s + 1);
    good = good && e > b && runs.slot_of(b) == s && runs.slot_of(e - 1) == s &&
           runs.slot_of(b + (e - b) / 2) == s;
    shortest = e - b < shortest ? e - b : shortest;
    longest = e - b > longest ? e - b : longest;
    ++g_runs;
  }
  // no run of a generation is longer than its weight's part by more than a unit
  good = good && longest <= 3 * ((long)shortest + 1);
  if (!good && ++g_bad <= 10) fprintf(stderr, "FAIL generations %d most %d units %d\n", GENS, most, units);
}

void check_all(int most, int units) {
  check<1>(most, units);
  check<2>(most, units);
  check<3>(most, units);
}

}  // namespace

int main() {
  for (int most = 1; most < 100; ++most)
    for (int units = 1; units < 700; units += units < 320 ? 1 : 13) check_all(most, units);
  std::mt19937 rng(7);
  for (int i = 0; i < 4000; ++i) {
    const int most = 1 + (int)(rng() % 768);
    const int bits = 1 + (int)(rng() % 31);
    check_all(most, 1 + (int)(rng() % ((1u << bits) - 1)));
    check_all(most, 0x7FFFFFFF - (int)(rng() % 5000));
  }
  printf("runs: %ld checked, %ld failure(s)\n", g_runs, g_bad);
  return g_bad ? 1 : 0;
}
