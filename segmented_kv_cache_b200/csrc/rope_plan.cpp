// The rotary plan (host): each pair's frequency, scaled, as a fraction of a turn per
// position in units of 2^-64.  Computed in long double, whose 64-bit mantissa the
// fraction can use where a double's 53 bits would not fill it.
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "seg_draft.h"

extern "C" int seg_attn_rope_plan(int rotary_dim, int layout, double base,
                                  const seg_attn_rope_scaling* scaling, seg_attn_rope_desc* desc) {
  if (!desc) return SEG_ATTN_ERR_INVALID_ARG;
  *desc = seg_attn_rope_desc{};
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > 2 * SEG_ATTN_ROPE_MAX_PAIRS)
    return SEG_ATTN_ERR_UNSUPPORTED;
  if (layout != SEG_ATTN_ROPE_HALF && layout != SEG_ATTN_ROPE_INTERLEAVED)
    return SEG_ATTN_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return SEG_ATTN_ERR_INVALID_ARG;
  const int kind = scaling ? scaling->kind : SEG_ATTN_ROPE_SCALE_NONE;
  const int pairs = rotary_dim / 2;
  const long double kTwoPi = 6.28318530717958647692528676655900577L;
  long double b = base, f = 1.0L, len = 1.0L, low = 1.0L, high = 1.0L;
  double amp = 1.0;
  if (kind < SEG_ATTN_ROPE_SCALE_NONE || kind > SEG_ATTN_ROPE_SCALE_PER_PAIR)
    return SEG_ATTN_ERR_INVALID_ARG;
  auto good = [](double x) { return x > 0.0 && std::isfinite(x); };
  if (kind != SEG_ATTN_ROPE_SCALE_NONE && kind != SEG_ATTN_ROPE_SCALE_PER_PAIR) {
    if (!good(scaling->factor)) return SEG_ATTN_ERR_INVALID_ARG;
    f = scaling->factor;
  }
  if (kind == SEG_ATTN_ROPE_SCALE_YARN || kind == SEG_ATTN_ROPE_SCALE_WAVELENGTH) {
    const bool unset = scaling->low == 0.0 && scaling->high == 0.0;
    low = unset ? 1.0 : scaling->low;
    high = unset ? (kind == SEG_ATTN_ROPE_SCALE_YARN ? 32.0 : 4.0) : scaling->high;
    if (!good(scaling->original_len) || !good((double)low) || !good((double)high) || !(low < high))
      return SEG_ATTN_ERR_INVALID_ARG;
    len = scaling->original_len;
  }
  if (kind == SEG_ATTN_ROPE_SCALE_NTK && rotary_dim > 2)
    b = b * powl(f, (long double)rotary_dim / (rotary_dim - 2));
  if (kind == SEG_ATTN_ROPE_SCALE_YARN) amp = (double)(0.1L * logl(f) + 1.0L);
  if (kind == SEG_ATTN_ROPE_SCALE_PER_PAIR) {
    if (!scaling->factors || scaling->num_factors != pairs) return SEG_ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < pairs; ++i)
      if (!good(scaling->factors[i])) return SEG_ATTN_ERR_INVALID_ARG;
  }
  if (scaling && scaling->amp != 0.0) amp = scaling->amp;
  if (!good(amp) || !std::isfinite((float)amp) || !((float)amp > 0.f))
    return SEG_ATTN_ERR_INVALID_ARG;
  long double ramp0 = 0.0L, ramp1 = 0.0L;  // YARN: pairs where the ramp starts and ends
  if (kind == SEG_ATTN_ROPE_SCALE_YARN) {
    auto pair = [&](long double turns) {
      return rotary_dim * logl(len / (turns * kTwoPi)) / (2.0L * logl(b));
    };
    ramp0 = std::min(std::max(floorl(pair(high)), 0.0L), (long double)(rotary_dim - 1));
    ramp1 = std::min(std::max(ceill(pair(low)), 0.0L), (long double)(rotary_dim - 1));
    if (ramp1 - ramp0 < 1e-3L) ramp1 = ramp0 + 1e-3L;
  }
  auto unit = [](long double x) { return std::min(std::max(x, 0.0L), 1.0L); };
  for (int i = 0; i < pairs; ++i) {
    long double w = powl(b, -2.0L * i / rotary_dim);
    if (kind == SEG_ATTN_ROPE_SCALE_LINEAR) {
      w /= f;
    } else if (kind == SEG_ATTN_ROPE_SCALE_YARN) {
      const long double r = unit((i - ramp0) / (ramp1 - ramp0));
      w = w * (1.0L - r) + w / f * r;
    } else if (kind == SEG_ATTN_ROPE_SCALE_WAVELENGTH) {
      const long double k = unit((len * w / kTwoPi - low) / (high - low));
      w = w * k + w / f * (1.0L - k);
    } else if (kind == SEG_ATTN_ROPE_SCALE_PER_PAIR) {
      w /= scaling->factors[i];
    }
    // whole turns per position change nothing at integer positions
    long double turn = w / kTwoPi;
    turn -= floorl(turn);
    const long double scaled = roundl(ldexpl(turn, 64));
    desc->turns[i] = scaled >= ldexpl(1.0L, 64) ? 0u : (uint64_t)scaled;
  }
  desc->magic = SEG_ATTN_ROPE_MAGIC;
  desc->rotary_dim = rotary_dim;
  desc->layout = layout;
  desc->amp = (float)amp;
  return SEG_ATTN_OK;
}
