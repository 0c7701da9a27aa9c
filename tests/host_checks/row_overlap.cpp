// Host-only check of dbs_rows_meet (the library's values.h, compiled for the host only; no GPU) against the sets of bytes.
//
// Claim: rows that share a byte are always found; with both strides alike, or with spans apart, others are never taken to meet.
#include <stdio.h>

#include <random>
#include <set>

#include "../../spmspv_graph_traversal_amd/csrc/values.h"

static std::set<long> bytes_of(const dbs_rows &r) {
  std::set<long> s;
  for (long i = 0; i < (long)r.ni; ++i)
    for (long j = 0; j < (long)r.nj; ++j)
      for (long d = 0; d < (long)r.width; ++d) s.insert((long)(r.at + i * r.si + j * r.sj) + d);
  return s;
}

int main() {
  std::mt19937 rng(1);
  const auto pick = [&](int low, int high) { return (int)(rng() % (unsigned)(high - low + 1)) + low; };
  long failures = 0, alike = 0, apart = 0, met = 0, one_alike = 0;
  for (int k = 0; k < 300000; ++k) {
    dbs_rows a = {pick(0, 60), pick(1, 4), pick(-20, 20), pick(1, 4), pick(-20, 20), pick(1, 6)}, b = a;
    b.at = pick(0, 60);
    b.width = pick(1, 6);
    const int kind = pick(0, 3);
    if (kind & 1) b.si = pick(-20, 20);
    if (kind & 2) b.sj = pick(-20, 20);
    const std::set<long> sa = bytes_of(a), sb = bytes_of(b);
    bool meet = false;
    for (long x : sa) meet |= sb.count(x) != 0;
    const bool answer = dbs_rows_meet(a, b);
    const bool like = (a.ni < 2 || a.si == b.si) && (a.nj < 2 || a.sj == b.sj);
    const bool spans = *sa.rbegin() >= *sb.begin() && *sb.rbegin() >= *sa.begin();
    if ((meet && !answer) || (!meet && answer && (like || !spans))) {
      if (++failures < 5) printf("FAIL case %d: %d, found %d\n", k, meet, answer);
    }
    met += meet;
    alike += like && spans && !meet;
    apart += !spans;
    one_alike += !like && spans && !meet && !answer;
  }
  // far apart and large: nothing wraps
  const __int128 big = (__int128)1 << 62;
  if (dbs_rows_meet({0, 1 << 30, big, 2, 5, 5}, {10, 1 << 30, big, 2, 5, 5}) || !dbs_rows_meet({0, 1 << 30, big, 2, 5, 6}, {10, 1 << 30, big, 2, 5, 5})) {
    ++failures;
    puts("FAIL large strides");
  }
  // four tokens from one row of 24 floats, out behind it
  if (dbs_rows_meet({0, 4, 0, 3, 32, 32}, {160, 4, 96, 3, 32, 32})) {
    ++failures;
    puts("FAIL out behind a row that is read four times");
  }
  printf("%ld met, %ld of like strides did not, %ld had spans apart, %ld one like stride; %ld failures\n", met, alike, apart, one_alike, failures);
  return failures != 0 || !met || !alike || !apart || !one_alike;
}
