// scan_order_harness.cpp -- the order in which the channelwise recurrence's workgroups
// take its tiles (turn_of in scan_kernels.h): every tile once, a tile after all that it
// waits for, and no tile for a number behind the last.  Built and run by
// tests/test_scan_order.py; nothing touches a GPU.
#include <cstdio>
#include <vector>

#include "scan_kernels.h"

using namespace gdr::scan;

static int check(int nchain, int nt, int team) {
  const uint32_t n = (uint32_t)nchain * nt;
  std::vector<uint32_t> number(n, n);
  for (uint32_t i = 0; i < n; ++i) {
    const Turn t = turn_of(i, nchain, nt, team);
    if (t.chain < 0 || t.chain >= nchain || t.tt < 0 || t.tt >= nt) return 1;
    uint32_t& at = number[(size_t)t.chain * nt + t.tt];
    if (at != n) return 2;
    at = i;
    if (t.tt > 0 && number[(size_t)t.chain * nt + t.tt - 1] >= i) return 3;   // n: not taken yet
  }
  for (uint32_t i : {n, n + 1, n + (uint32_t)team, 2 * n, 3 * n + 7, 0xffffffffu})
    if (i >= n && turn_of(i, nchain, nt, team).chain != -1) return 4;
  return 0;
}

int main() {
  for (int team : {team_of(true, GDR_BF16), team_of(false, GDR_BF16)})
    for (int nchain : {1, 2, 31, 32, 33, 47, 64, 100, 127, 128, 129, 200, 300})
      for (int nt : {1, 2, 3, 7, 8, 9, 17, 64, 65}) {
        const int r = check(nchain, nt, team);
        if (r) return std::printf("chains %d, tiles %d, team %d: %d\n", nchain, nt, team, r), 1;
      }
  // the most tiles of a launch, in few chains and in many
  const int most = (int)kMaxTiles - 1;
  for (int team : {32, 128})
    for (int nchain : {1, 37, 4096, most}) {
      const int nt = most / nchain;
      const Turn t = turn_of((uint32_t)nchain * nt - 1, nchain, nt, team);
      if (t.chain != nchain - 1 || t.tt != nt - 1) return std::printf("last of %d x %d\n", nchain, nt), 1;
      if (turn_of((uint32_t)nchain * nt, nchain, nt, team).chain != -1) return 1;
    }
  std::printf("SCAN_ORDER_OK\n");
  return 0;
}
