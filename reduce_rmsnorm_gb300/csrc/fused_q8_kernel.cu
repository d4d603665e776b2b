// The fused step with its output in e4m3 with scales: the instances of
// fused_forms.cuh whose rows end in 8 bits, and the rule that hands some row
// lengths to the combine step's ring.
#define TW_FUSED_Q8 1
#include "fused_forms.cuh"

namespace tw {

namespace {

// Whether the combine step's ring, without slots, serves this launch: it puts
// several CTAs on an SM, each with a row at a time, where the forms here have
// one. For short rows of whole-GPU launches that are too many for the direct
// form, where one CTA's pace over a row, not HBM, is the bound. Measured here
// against there (T = 1200 / 4000): N = 1, H = 264 9.3 / 27.1 against 4.2 / 7.2
// us; N = 3, H = 1152 10.3 / 31.9 against 5.2 / 13.8; N = 8, H = 4096 18.6 /
// 54.2 against 16.4 / 54.3; N = 14, H = 4096 24.4 / 72.2 against 24.7 / 72.7.
// Of the rows over 2048 that leave threads idle the shorter ones stay here (N =
// 3, H = 2816 14.9 / 39.3 against 14.5 / 43.3, H = 5000 19.4 / 57.1 against 18.0
// / 55.1, 7.0 against 8.0 at T = 333); those over 8192, whose instances here
// spill, go there as well (N = 3, H = 12000 47.8 / 147.7 against 36.0 / 112.0,
// N = 8, H = 16000 82.5 / 235.9 against 67.3 / 220.2).
bool use_shared_ring(const FusedArgs& a, int sm_budget) {
  const bool shorter = (a.hidden <= 2048 || a.hidden == 4096) && (a.n + 1) * a.hidden <= 36864;
  const bool longer = a.hidden > 8192 && a.hidden < 16384 && a.n <= 12;
  if (sm_budget != 0 || !(shorter || longer)) return false;
  DeviceInfo* d = nullptr;
  Choice c;
  LaunchShape shape;
  return device_info(&d) == TW_OK && a.rows > d->sms &&
         shape_for(*d, a.rows, a.hidden, a.n, 0, &c, &shape) == TW_OK && !c.direct;
}

}  // namespace

int launch_fused_q8(const FusedArgs& a, cudaStream_t stream, int sm_budget) {
  if (!use_shared_ring(a, sm_budget)) return launch_forms(a, stream, sm_budget, nullptr);
  CombineArgs c = {};
  for (int r = 0; r < a.n; ++r) c.partials[r] = a.partials[r];
  c.n = a.n;
  c.residual = a.residual;
  c.gamma = a.gamma;
  c.out = a.out;
  c.scales = a.scales;
  c.group = a.group;
  c.scale_type = a.scale_type;
  c.eps = a.eps;
  c.tokens = a.rows;
  c.hidden = a.hidden;
  return launch_combine(c, stream, 0);
}

int read_fused_q8_error(int reset, unsigned* code) { return read_ring_error(reset, code); }

}  // namespace tw
