"""What the compiler is told of pointers that a call allows to be the same (no GPU): nothing."""
import os
import re
import subprocess

import pytest

from sigmoid_top_routing_02_amd import build as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.HIPCC), reason="hipcc not found")

# source, kernel, parameters that may overlap: dz_q is z_q and dz_scale z_scale; dlogits is dlogits_in; de is de_in
OVERLAPS = [("backward.hip", "swiglu_backward_zq_kernel", (0, 1, 5, 6)), ("balance.hip", "balance_backward_kernel", (9, 10)),
            ("logits.hip", "logits_sum_kernel", (3, 4))]


@pytest.mark.parametrize("source,kernel,which", OVERLAPS)
def test_overlapping_arguments_are_not_declared_apart(source, kernel, which):
    flags = [f for f in b.flags_of(source) if f != "-shared"]
    r = subprocess.run([b.HIPCC, *flags, "-I", os.path.join(b.ROOT, "include"), "--cuda-device-only", "-S", "-emit-llvm",
                        "-o", "-", os.path.join(b.CSRC, source)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    heads = re.findall(r"^define [^\n]*@\S*\d" + kernel + r"\w*\(([^\n]*)\) [^\n(]*\{$", r.stdout, re.M)
    assert heads, kernel
    for head in heads:
        # commas inside an attribute's brackets do not part parameters
        params = re.sub(r"\([^()]*\)", "", head).split(", ")
        for i in which:
            assert params[i].startswith("ptr ") and "noalias" not in params[i], (kernel, i, params[i])
