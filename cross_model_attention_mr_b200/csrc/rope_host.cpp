// mr_rope_init: the position step of every rotated pair, as a 64-bit fraction of a turn.
#include <math.h>
#include <stdint.h>

#include "../../include/mr.h"

extern "C" mr_status mr_rope_init(mr_rope* out, int d, int rot_dim, int interleaved, double base,
                                  mr_rope_scaling scaling, double factor, int orig_len, double beta_slow,
                                  double beta_fast, double mscale, const double* inv_freq) {
  if (!out || d < 8 || d > 256 || d % 8 || rot_dim < 2 || rot_dim > d || rot_dim % 2) return MR_ERR_INVALID_ARG;
  if (!isfinite(mscale) || !isfinite((float)mscale)) return MR_ERR_INVALID_ARG;
  // extended precision throughout: a relative error of 2^-53 in f_i alone would show at the longest positions
  const long double two_pi = 6.283185307179586476925286766559005768L;
  if (!inv_freq) {
    if (!(base > 1.0) || !isfinite(base) || !(factor > 0.0) || !isfinite(factor)) return MR_ERR_INVALID_ARG;
    switch (scaling) {
      case MR_ROPE_NONE:
        if (factor != 1.0) return MR_ERR_INVALID_ARG;
        break;
      case MR_ROPE_LINEAR: break;
      case MR_ROPE_BASE:
        if (rot_dim < 4) return MR_ERR_INVALID_ARG;
        break;
      case MR_ROPE_RAMP:
        if (orig_len < 1 || !(beta_slow >= 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast))
          return MR_ERR_INVALID_ARG;
        break;
      default: return MR_ERR_INVALID_ARG;
    }
  }
  mr_rope r = {};
  r.d = d;
  r.rot_dim = rot_dim;
  r.interleaved = interleaved ? 1 : 0;
  r.mscale = (float)mscale;
  long double b = base;
  if (!inv_freq && scaling == MR_ROPE_BASE) b *= powl((long double)factor, (long double)rot_dim / (rot_dim - 2));
  for (int i = 0; i < rot_dim / 2; ++i) {
    long double f;
    if (inv_freq) {
      if (!isfinite(inv_freq[i])) return MR_ERR_INVALID_ARG;
      f = inv_freq[i];
    } else {
      f = powl(b, -(long double)(2 * i) / rot_dim);
      if (scaling == MR_ROPE_LINEAR) f /= factor;
      if (scaling == MR_ROPE_RAMP) {
        const long double turns = orig_len * f / two_pi;
        long double g = (turns - beta_slow) / ((long double)beta_fast - beta_slow);
        g = g < 0 ? 0 : g > 1 ? 1 : g;
        f = g * f + (1 - g) * f / factor;
      }
    }
    const long double t = fabsl(f) / two_pi;
    if (!(t < 1.0L)) return MR_ERR_INVALID_ARG;  // one turn per position or more
    const long double scaled = t * 18446744073709551616.0L + 0.5L;
    const uint64_t u = scaled >= 18446744073709551615.0L ? UINT64_MAX : (uint64_t)scaled;
    r.turn[i] = f < 0 ? (uint64_t)0 - u : u;
  }
  *out = r;
  return MR_OK;
}
