// One row of the clipped policy loss, shared by the loss on given logits, the
// loss on per-row log-probabilities and the fused head's combine step.
#pragma once

#include <cstddef>

namespace flce {

struct PolicyArgs {
  const float* old_logp;  // [N] or null: the current log-probabilities themselves (r = 1)
  const float* adv;       // [N]
  const float* ref_logp;  // [N] or null: no KL term
  double lo, hi;          // 1 - clip_low, 1 + clip_high
  double kl_coef;
};

struct PolicyRow {
  double loss, dlogp, kl;
};

// A row's inputs, loaded ahead of the log-probability that they meet.
struct PolicyIn {
  float old, adv, ref;
};
__device__ __forceinline__ PolicyIn policy_load(const PolicyArgs& p, size_t row) {
  return {p.old_logp ? p.old_logp[row] : 0.f, p.adv[row], p.ref_logp ? p.ref_logp[row] : 0.f};
}

// One row's policy loss (without an entropy term), its derivative by lp and the
// KL estimate, in fp64: the ratio is compared with the clip borders, where a
// rounding would switch the row's gradient on or off, and the KL estimate is a
// small difference.  Written so that a clipped-away infinite ratio gives the
// border's value and a NaN stays a NaN.
__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& p, const PolicyIn& in, double lp) {
  PolicyRow o;
  const double A = static_cast<double>(in.adv);
  const double r = p.old_logp ? exp(lp - static_cast<double>(in.old)) : 1.0;
  const bool clipped = A >= 0.0 ? r > p.hi : r < p.lo;
  const double rc = !clipped ? r : A >= 0.0 ? p.hi : p.lo;
  o.loss = -A * rc;
  o.dlogp = clipped ? 0.0 : o.loss;
  o.kl = 0.0;
  if (p.ref_logp) {
    const double d = static_cast<double>(in.ref) - lp;
    const double em1 = expm1(d);
    o.kl = isinf(em1) ? em1 : em1 - d;  // lp = -infinity: the estimate's limit, not infinity less infinity
    if (p.kl_coef != 0.0) {
      o.loss += p.kl_coef * o.kl;
      o.dlogp -= p.kl_coef * em1;
    }
  }
  return o;
}

}  // namespace flce
