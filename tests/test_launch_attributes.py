"""Every programmatic dependent launch is configured in one place, which BSF_DISABLE_PDL turns into ordinary
launches, those in clusters too.  CPU-only: the configurations are built, nothing is launched."""

import os
import re
import subprocess

import pytest

from block_scaled_fp8_route_gb300 import build

CSRC = os.path.join(os.path.dirname(build.__file__), "csrc")
PROGRAM = r"""
#include <cstdio>
#include "host_utils.h"
int main() {
  for (unsigned cluster : {0u, 1u, 2u, 8u}) {
    bsf::DependentLaunch l(dim3(16, 3), 256, 1000, nullptr, cluster);
    unsigned size = 0, dependent = 0;
    for (unsigned i = 0; i < l.cfg.numAttrs; ++i) {
      if (l.cfg.attrs[i].id == cudaLaunchAttributeClusterDimension) size = l.cfg.attrs[i].val.clusterDim.x;
      if (l.cfg.attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization)
        dependent = l.cfg.attrs[i].val.programmaticStreamSerializationAllowed;
    }
    std::printf("%u %u %u %u %u %zu\n", size, dependent, l.cfg.numAttrs, l.cfg.gridDim.x * l.cfg.gridDim.y,
                l.cfg.blockDim.x, l.cfg.dynamicSmemBytes);
  }
}
"""


@pytest.mark.parametrize("disabled", [False, True])
def test_configurations(tmp_path, disabled):
    src, exe = tmp_path / "launch.cu", tmp_path / "launch"
    src.write_text(PROGRAM)
    flags = [f for f in build.NVCC_FLAGS if f != "-lineinfo"] + ["-I" + CSRC] + ["-DBSF_DISABLE_PDL"] * disabled
    subprocess.run([build._nvcc(), *flags, str(src), "-o", str(exe)], check=True, capture_output=True)
    rows = [[int(v) for v in line.split()] for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                                      text=True).stdout.splitlines()]
    on = 0 if disabled else 1
    assert rows == [[size, on, on + (size > 0), 48, 256, 1000] for size in (0, 1, 2, 8)]


def test_no_other_place_sets_the_attribute():
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert name == "host_utils.h" or "ProgrammaticStreamSerialization" not in text, name
