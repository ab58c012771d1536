"""CPU tier: every documented build option of the Newton-Schulz GEMMs still compiles for gfx950."""
import os
import subprocess

import pytest

pytest.importorskip("torch")


@pytest.mark.parametrize("option", [None, "HPO_NS_GEN_HALF=1", "HPO_NS_XBAR=0", "HPO_NS_SCHED=0", "HPO_NS_PRIO=0",
                                    "HPO_NS_GROUP=0"])
def test_muon_kernels_compile_with(option):
    from mixed_precision_optimizer_amd import build
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc here")
    cmd = [cc, *build.DEVICE_FLAGS, "--cuda-device-only", "-fsyntax-only", "-I", build.INCLUDE, "-I", build.CSRC,
           os.path.join(build.CSRC, "hpo_muon.hip")] + ([f"-D{option}"] if option else [])
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
