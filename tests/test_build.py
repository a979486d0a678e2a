"""What the compiler says of the sources, and what it is told of addresses (no GPU)."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from sigmoid_top_routing_02_amd import build as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.HIPCC), reason="hipcc not found")


def _compile(source, *extra):
    flags = [f for f in b.flags_of(source) if f != "-shared"]
    return subprocess.run([b.HIPCC, *flags, "-I", os.path.join(b.ROOT, "include"), *extra, source],
                          capture_output=True, text=True)


def test_sources_compile_without_warnings():
    with ThreadPoolExecutor(max_workers=8) as ex:
        for source, r in zip(b.sources(), ex.map(lambda s: _compile(s, "-fsyntax-only"), b.sources())):
            said = [line for line in r.stderr.splitlines() if "warning:" in line]
            assert r.returncode == 0 and not said, f"{os.path.basename(source)}: {said}"


def test_unaligned_rows_are_accessed_at_their_own_alignment():
    """In the norm's kernels for rows that start off 16 bytes (the second template argument false), every
    vector access of device memory promises the values' alignment at most: 4 bytes, or 2 for bf16."""
    r = _compile(os.path.join(b.CSRC, "norm.hip"), "--cuda-device-only", "-S", "-emit-llvm", "-o", "-")
    assert r.returncode == 0, r.stderr
    kernels = re.findall(r"^define [^\n]*@(\S*add_rmsnorm\w*kernelILi\dELb0E\w*)\([^\n]*\{\n(.*?)^\}", r.stdout, re.S | re.M)
    assert len(kernels) >= 6, [name for name, _ in kernels]
    for name, body in kernels:
        aligns = {"load": set(), "store": set()}
        for line in body.splitlines():
            m = re.search(r"\b(load|store) <\d+ x (?:float|i32|i16)>.*addrspace\(1\).*align (\d+)", line)
            if m:
                aligns[m.group(1)].add(int(m.group(2)))
        assert aligns["load"] and aligns["store"], name
        assert aligns["load"] <= {2, 4} and aligns["store"] <= {2, 4}, (name, aligns)
