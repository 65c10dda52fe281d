"""The window attention's mask in 32 x 32 tiles, evaluated by the compiler as constants at its borders (no GPU needed): an
integer overflow is no constant expression, and a wrong value fails its assertion."""
import os
import subprocess

import pytest

from selective_state_space_03_amd import build

# queries of a tile of 128: their least and greatest positions (those of more queries than keys are negative)
HEAD = """
#include "attn_device.h"
using namespace ssm;
constexpr bool seen(int pos, int j0, int h, int j, int window, int sinks) {
  const WideMask m = wide_mask(pos, j0, h, window, sinks);
  return j <= m.d && (j > m.w || j < m.f);
}
// a tile that is not there: no key of it is seen by any query of the wave
constexpr bool none(int p0, int window, int sinks) {
  for (int c = 0; c < 32; ++c)
    for (int h = 0; h < 2; ++h)
      for (int e = 0; e < 64; ++e)
        if (seen(p0 + c, NONE(p0), h, 8 * (e / 4) + e % 4, window, sinks)) return false;
  return true;
}
constexpr int kLast = kAttnAll - 1;
static_assert(none(0, kAttnAll, 0) && none(-127, kAttnAll, 0) && none(-127, 1, 0) && none(kLast - 31, kAttnAll, 0));
static_assert(none(0, 1024, 1024) && none(5000, 1024, 4) && none(-96, 1500, 1400));
// the first and the last key of the longest sequence, with and without a window
static_assert(seen(kLast, 0, 0, 0, kAttnAll, 0) && seen(kLast, kLast - 63, 0, 63, kAttnAll, 0) && !seen(kLast - 1, kLast - 63, 0, 63, kAttnAll, 0));
static_assert(!seen(kLast, 0, 0, 0, kLast, 0) && seen(kLast, 0, 0, 1, kLast, 0) && seen(kLast, 0, 0, 0, kLast, 1));
static_assert(!seen(-1, 0, 0, 0, kAttnAll, 0) && seen(0, 0, 0, 0, kAttnAll, 0) && !seen(-128, 0, 1, 0, kAttnAll, 0));
"""


def _compiles(none, tmp_path):
    src = tmp_path / "mask.hip"
    src.write_text(HEAD.replace("NONE(p0)", none))
    cmd = [build.hipcc(), "-std=c++17", "-fsyntax-only", "--offload-host-only", f"--offload-arch={build.ARCH}", "-I", build.INCLUDE, "-I",
           build.CSRC, str(src)]
    return subprocess.run(cmd, capture_output=True, text=True, env=dict(os.environ))


def test_the_mask_at_its_borders(tmp_path):
    r = _compiles("wide_none(p0)", tmp_path)
    assert r.returncode == 0, r.stderr[-3000:]


@pytest.mark.parametrize("none", ["kAttnAll"])
def test_the_compiler_sees_an_overflow(none, tmp_path):
    """The longest sequence's length in the place of a tile that is not there leaves 32 bits without a window."""
    r = _compiles(none, tmp_path)
    assert r.returncode != 0 and "outside the range of representable values" in r.stderr
