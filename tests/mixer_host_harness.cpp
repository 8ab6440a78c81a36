// mixer_host_harness.cpp -- the host half of the convolution, the selective scan and the
// gated group norm (argument checks) under AddressSanitizer and UndefinedBehaviorSanitizer.
// The launchers are replaced by recorders, so nothing touches a GPU; the pointers are fake
// and never dereferenced.  Built and run by tests/test_abi_mixer.py.
#include <cstdio>
#include <cstdlib>

#include "conv_kernels.h"
#include "gnorm_kernels.h"
#include "ssm_kernels.h"

static int g_launches = 0;

namespace gdr {
namespace conv {
size_t bwd_workspace(int, int, int, int) { return 4096; }
hipError_t launch_conv_fwd(const gdr_conv_args&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_conv_bwd(const gdr_conv_bwd_args&, hipStream_t) { return ++g_launches, hipErrorInvalidValue; }
hipError_t launch_conv_step(const gdr_conv_step_args&, hipStream_t) { return ++g_launches, hipSuccess; }
}  // namespace conv
namespace ssm {
size_t fwd_workspace(int, int, int, int, int) { return 4096; }
size_t bwd_workspace(int, int, int, int, int, bool) { return 4096; }
hipError_t launch_ssm_fwd(const gdr_ssm_args&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_ssm_bwd(const gdr_ssm_bwd_args&, hipStream_t) { return ++g_launches, hipErrorInvalidValue; }
hipError_t launch_ssm_step(const gdr_ssm_step_args&, hipStream_t) { return ++g_launches, hipSuccess; }
}  // namespace ssm
namespace gnorm {
size_t bwd_workspace(int64_t, int, int, int) { return 4096; }
hipError_t launch_gnorm_fwd(const gdr_gnorm_args&, hipStream_t) { return ++g_launches, hipSuccess; }
hipError_t launch_gnorm_bwd(const gdr_gnorm_bwd_args&, hipStream_t) { return ++g_launches, hipErrorInvalidValue; }
}  // namespace gnorm
}  // namespace gdr

// far apart, 16-byte aligned
static char* at(int i) { return reinterpret_cast<char*>((uintptr_t)(i + 1) << 48); }

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
  gdr_conv_args f{};
  f.B = 1, f.T = (1 << 30) - 1, f.C = 1, f.K = 8, f.io_dtype = GDR_F32;
  f.x = at(0), f.weight = (float*)at(1), f.y = at(2), f.state = at(3), f.state_out = at(3);
  EXPECT(gdr_conv_fwd(&f, nullptr), GDR_ERR_UNSUPPORTED);   // workgroups
  f.T = 256 * ((1 << 22) - 1);
  EXPECT(gdr_conv_fwd(&f, nullptr), GDR_OK);
  f.B = 1 << 15, f.T = (1 << 15) - 1;
  EXPECT(gdr_conv_fwd(&f, nullptr), GDR_ERR_UNSUPPORTED);   // 2^15 x 128
  f.T = 127 * 256;
  EXPECT(gdr_conv_fwd(&f, nullptr), GDR_OK);
  f.B = f.T = f.C = 2147483647;
  EXPECT(gdr_conv_fwd(&f, nullptr), GDR_ERR_UNSUPPORTED);
  f.C = 1;
  EXPECT(gdr_conv_fwd(&f, nullptr), GDR_ERR_SHAPE);

  gdr_conv_bwd_args b{};
  b.B = 3, b.T = 100, b.C = 130, b.K = 4, b.io_dtype = GDR_BF16;
  b.x = at(0), b.weight = (float*)at(1), b.grad_y = at(2), b.grad_x = at(3), b.grad_weight = (float*)at(4);
  EXPECT(gdr_conv_bwd(&b, nullptr), GDR_ERR_WORKSPACE);
  b.workspace = at(5), b.workspace_bytes = 4095;
  EXPECT(gdr_conv_bwd(&b, nullptr), GDR_ERR_WORKSPACE);
  b.workspace_bytes = 4096;
  EXPECT(gdr_conv_bwd(&b, nullptr), GDR_ERR_HIP);           // a failed launch
  if (gdr_conv_bwd_workspace(&b) != 4096) return 1;
  b.grad_x = at(2) + 2;                                     // overlaps grad_y
  EXPECT(gdr_conv_bwd(&b, nullptr), GDR_ERR_ARG);
  if (gdr_conv_bwd_workspace(&b) != 0) return 1;

  gdr_conv_step_args c{};
  c.N = 1 << 21, c.C = 1024, c.K = 2, c.io_dtype = GDR_BF16;
  c.x = at(0), c.weight = (float*)at(1), c.state = at(2), c.state_out = at(2), c.y = at(3);
  EXPECT(gdr_conv_step(&c, nullptr), GDR_ERR_SHAPE);
  c.N -= 1;
  EXPECT(gdr_conv_step(&c, nullptr), GDR_OK);
  c.K = 4;
  EXPECT(gdr_conv_step(&c, nullptr), GDR_ERR_SHAPE);

  gdr_ssm_args s{};
  s.B = 1 << 22, s.T = 1, s.C = 64, s.N = 64, s.G = 1, s.io_dtype = GDR_F32;
  s.x = at(0), s.dt = at(1), s.A = (float*)at(2), s.Bv = at(3), s.Cv = at(4), s.y = at(5);
  s.workspace = at(6), s.workspace_bytes = 4096;
  EXPECT(gdr_ssm_fwd(&s, nullptr), GDR_ERR_UNSUPPORTED);    // chains
  s.B -= 1;
  EXPECT(gdr_ssm_fwd(&s, nullptr), GDR_OK);
  s.C = 65;
  EXPECT(gdr_ssm_fwd(&s, nullptr), GDR_ERR_UNSUPPORTED);
  s.B = s.T = 2147483647;
  EXPECT(gdr_ssm_fwd(&s, nullptr), GDR_ERR_SHAPE);

  gdr_ssm_bwd_args t{};
  t.B = 2, t.T = 100, t.C = 130, t.N = 16, t.G = 2, t.io_dtype = GDR_BF16;
  t.x = at(0), t.dt = at(1), t.A = (float*)at(2), t.Bv = at(3), t.Cv = at(4), t.grad_y = at(5);
  t.grad_x = at(6), t.grad_dt = at(7), t.grad_A = (float*)at(8), t.grad_Bv = at(9), t.grad_Cv = at(10);
  EXPECT(gdr_ssm_bwd(&t, nullptr), GDR_ERR_WORKSPACE);
  t.workspace = at(11), t.workspace_bytes = 4096;
  EXPECT(gdr_ssm_bwd(&t, nullptr), GDR_ERR_HIP);
  t.grad_Cv = at(9) + 2;
  EXPECT(gdr_ssm_bwd(&t, nullptr), GDR_ERR_ARG);
  if (gdr_ssm_bwd_workspace(&t) != 0) return 1;

  gdr_ssm_step_args u{};
  u.R = 1 << 15, u.C = 1 << 10, u.N = 64, u.G = 1, u.io_dtype = GDR_F32;
  u.x = at(0), u.dt = at(1), u.A = (float*)at(2), u.Bv = at(3), u.Cv = at(4), u.y = at(5);
  u.h = (float*)at(6), u.h_out = (float*)at(6);
  EXPECT(gdr_ssm_step(&u, nullptr), GDR_ERR_SHAPE);
  u.R -= 1;
  EXPECT(gdr_ssm_step(&u, nullptr), GDR_OK);

  gdr_gnorm_args n{};
  n.R = (1LL << 30), n.C = 4, n.G = 2, n.io_dtype = GDR_BF16, n.center = 1, n.eps = 1e-5f;
  n.x = at(0), n.y = at(1);
  EXPECT(gdr_gnorm_fwd(&n, nullptr), GDR_ERR_SHAPE);
  n.R -= 1;
  EXPECT(gdr_gnorm_fwd(&n, nullptr), GDR_OK);
  n.R = (1LL << 62), n.G = 4;
  EXPECT(gdr_gnorm_fwd(&n, nullptr), GDR_ERR_SHAPE);

  gdr_gnorm_bwd_args m{};
  m.R = 10, m.C = 64, m.G = 4, m.io_dtype = GDR_F32;
  m.x = at(0), m.rstd = (float*)at(1), m.grad_y = at(2), m.grad_x = at(3);
  EXPECT(gdr_gnorm_bwd(&m, nullptr), GDR_ERR_HIP);          // no columns' sums, no workspace
  m.grad_weight = (float*)at(4);
  EXPECT(gdr_gnorm_bwd(&m, nullptr), GDR_ERR_WORKSPACE);
  m.workspace = at(5), m.workspace_bytes = 4096;
  EXPECT(gdr_gnorm_bwd(&m, nullptr), GDR_ERR_HIP);
  if (g_launches != 10) return 2;
  std::printf("MIXER_HARNESS_OK\n");
  return 0;
}
