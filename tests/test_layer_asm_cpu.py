"""The inline assembly of the selective scan's lane sums, compiled for gfx950 and read back (CPU only):
it writes its in/out registers before it has read all of its inputs, so none of the inputs may share
a register with them, also where the compiler knows two values to be equal."""
import os
import re
import subprocess

import pytest

from bilinear_rnn_amd import build

# Every input equals an in/out value, as the compiler can see: the case in which it may use one register for both.
SOURCE = """
#include "scan_common.h"
namespace comba {
__global__ void equal_inputs(const float* in, float* out) {
  float v[4 * %(n)d];
  for (int i = 0; i < %(n)d; ++i) {
    const float x = in[threadIdx.x + 64 * i];
    for (int k = 0; k < 4; ++k) v[i + %(n)d * k] = x;
  }
  halve_bits_3_2<%(n)d>(v);
  for (int i = 0; i < %(n)d; ++i) out[threadIdx.x + 64 * i] = v[i];
}
}
"""


def asm_blocks(n, tmp_path):
    src, out = tmp_path / "lane_sums.hip", tmp_path / "lane_sums.s"
    src.write_text(SOURCE % dict(n=n))
    subprocess.run([build._hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S", str(src), "-o", str(out)],
                   check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    return re.findall(r"#ASMSTART(.*?)#ASMEND", out.read_text(), flags=re.S)


@pytest.mark.parametrize("n", [1, 2, 4, 8])   # 1: the other form
def test_inputs_share_no_register_with_what_is_written_before_them(n, tmp_path):
    blocks = [b for b in asm_blocks(n, tmp_path) if "v_add_f32_dpp" in b]
    assert len(blocks) == max(1, n // 2)
    for block in blocks:
        adds = [re.match(r"\s*v_add_f32_dpp (v\d+), (v\d+), (v\d+) ", line) for line in block.splitlines()
                if "v_add_f32_dpp" in line]
        assert len(adds) == (6 if n == 1 else 12) and all(adds), block
        # the first bit's additions come in pairs: A += A over the lanes, then A += B
        over8 = [m.groups() for m in adds[:4 if n == 1 else 8]]
        written, read = [a for a, _, _ in over8[::2]], [b for _, b, _ in over8[1::2]]
        assert len(set(written)) == len(written), block
        assert not set(written) & set(read), block
