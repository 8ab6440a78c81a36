// channelwise_host_harness.cpp -- the host half of the channelwise operators
// (argument checks in scan_api.cpp and norm_api.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer.  The launchers are replaced by recorders, so nothing
// touches a GPU; the pointers are fake and never dereferenced.  Built and run by
// tests/test_abi_channelwise.py.
#include <cstdio>
#include <cstdlib>

#include "norm_kernels.h"
#include "scan_kernels.h"

static int g_launches = 0;

namespace gdr {
namespace scan {
size_t fwd_workspace(int, int, int) { return 4096; }
size_t bwd_workspace(int, int, int, bool, bool) { return 4096; }
hipError_t launch_scan_fwd(const gdr_scan_args&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_scan_bwd(const gdr_scan_bwd_args&, hipStream_t) { return ++g_launches, hipErrorInvalidValue; }
hipError_t launch_scan_step(const gdr_scan_step_args&, hipStream_t) { return ++g_launches, hipSuccess; }
}  // namespace scan
namespace norm {
size_t bwd_workspace(int64_t, int) { return 4096; }
hipError_t launch_norm_fwd(const gdr_norm_args&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_norm_bwd(const gdr_norm_bwd_args&, hipStream_t) { return ++g_launches, hipSuccess; }
}  // namespace norm
namespace ckpt8 {
hipError_t launch_pack(const gdr_ckpt8_pack_args&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_unpack(const gdr_ckpt8_unpack_args&, hipStream_t) { return ++g_launches, hipSuccess; }
}  // namespace ckpt8
}  // namespace gdr

// far apart, 16-byte aligned
static char* at(int i) { return reinterpret_cast<char*>((uintptr_t)(i + 1) << 44); }

#define EXPECT(call, status)                                                          \
  do {                                                                                \
    const gdr_status got = (call);                                                    \
    if (got != (status)) {                                                            \
      std::fprintf(stderr, "line %d: status %d, expected %d\n", __LINE__, got, status); \
      return 1;                                                                       \
    }                                                                                 \
  } while (0)

int main() {
  // the largest sizes that the checks let through, and the first that they do not
  gdr_scan_args f{};
  f.B = 1;
  f.T = (1 << 22) - 1;
  f.C = 1 << 18;
  f.io_dtype = GDR_F32;
  f.x = at(0);
  f.alpha = (float*)at(1);
  f.y = at(2);
  f.workspace = at(3);
  f.workspace_bytes = 4096;
  EXPECT(gdr_scan_fwd(&f, nullptr), GDR_ERR_UNSUPPORTED);   // tiles
  f.T = 1 << 22;
  EXPECT(gdr_scan_fwd(&f, nullptr), GDR_ERR_SHAPE);
  f.T = 128 * 2047;
  EXPECT(gdr_scan_fwd(&f, nullptr), GDR_OK);
  f.T += 1;
  EXPECT(gdr_scan_fwd(&f, nullptr), GDR_ERR_UNSUPPORTED);
  f.B = f.T = f.C = 2147483647;
  EXPECT(gdr_scan_fwd(&f, nullptr), GDR_ERR_UNSUPPORTED);
  f.C = 1;
  EXPECT(gdr_scan_fwd(&f, nullptr), GDR_ERR_SHAPE);

  gdr_scan_bwd_args b{};
  b.B = 3;
  b.T = 100;
  b.C = 130;
  b.io_dtype = GDR_BF16;
  b.x = at(0);
  b.x_exp = (uint8_t*)at(1);
  b.decay_x = at(2);
  b.decay_a = (float*)at(3);
  b.grad_y = at(4);
  b.grad_x = at(5);
  b.grad_decay_x = at(6);
  b.grad_decay_a = (float*)at(7);
  EXPECT(gdr_scan_bwd(&b, nullptr), GDR_ERR_WORKSPACE);
  b.workspace = at(8);
  b.workspace_bytes = 4095;
  EXPECT(gdr_scan_bwd(&b, nullptr), GDR_ERR_WORKSPACE);
  b.workspace_bytes = 4096;
  EXPECT(gdr_scan_bwd(&b, nullptr), GDR_ERR_HIP);   // a failed launch
  if (gdr_scan_bwd_workspace(&b) != 4096) return 1;
  b.grad_x = (char*)at(4) + 2;                      // overlaps grad_y
  EXPECT(gdr_scan_bwd(&b, nullptr), GDR_ERR_ARG);
  if (gdr_scan_bwd_workspace(&b) != 0) return 1;

  gdr_norm_args n{};
  n.R = (1LL << 31) - 1;
  n.D = 512;
  n.io_dtype = GDR_BF16;
  n.x = at(0);
  n.y = at(1);
  EXPECT(gdr_norm_fwd(&n, nullptr), GDR_OK);
  n.D = 513;
  EXPECT(gdr_norm_fwd(&n, nullptr), GDR_ERR_SHAPE);
  n.R = INT64_MAX;
  EXPECT(gdr_norm_fwd(&n, nullptr), GDR_ERR_SHAPE);
  gdr_ckpt8_pack_args p{};
  p.R = 1023;
  p.D = 1 << 30;
  p.io_dtype = GDR_F32;
  p.x = at(0);
  p.code = (uint8_t*)at(1);
  p.exp = (uint8_t*)at(2);
  EXPECT(gdr_ckpt8_pack(&p, nullptr), GDR_OK);
  p.R = 1024;
  EXPECT(gdr_ckpt8_pack(&p, nullptr), GDR_ERR_SHAPE);
  if (g_launches != 4) return 1;
  std::puts("CHANNELWISE_HARNESS_OK");
  return 0;
}
