"""The rings of LDS buffers that memory-to-LDS loads refill, read from the
compiler's listing of the kernels (no GPU).

A wave gives a buffer up at a barrier; another wave's load may write into it
from there on. So before such a barrier the wave waits for its own reads of LDS
(lgkmcnt(0)) as well as for its loads, and the sources say so, instead of
leaving it to where the compiler puts the products that use the fragments. (At
a barrier of its own the compiler keeps account of them.)
"""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _build_module():
    # by path: importing the package would load the library, and with it a HIP
    # runtime, before the GPU tests of the same run load torch's
    spec = importlib.util.spec_from_file_location("lq_build", os.path.join(ROOT, "quantized_lora_fine_lq_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


build = _build_module()

KERNELS = {"lq_adapters.hip": ["k_adapter_down_tiles"],
           "lq_adapter_gemm.hip": ["k_adapter_gemm_small", "k_adapter_gemm"]}


@pytest.fixture(scope="module", params=sorted(KERNELS))
def functions(request, tmp_path_factory):
    """{mangled name: [(instruction, whether the source wrote it)]} of one source's ring kernels."""
    src = request.param
    out = tmp_path_factory.mktemp("asm") / (src + ".s")
    cmd = [build.hipcc(), f"--offload-arch={build.ARCH}", "-x", "hip", "-O3", "-std=c++17", "-ffp-contract=off",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-S", "--cuda-device-only",
           os.path.join(build.CSRC, src), "-o", str(out)]
    subprocess.run(cmd, check=True, capture_output=True)
    bodies, body, inline = {}, None, False
    for line in out.read_text().splitlines():
        inline = (inline or "#ASMSTART" in line) and "#ASMEND" not in line
        text = line.split(";")[0].strip()
        start = re.match(r"^(_Z\w+):", line)
        if start:
            name = re.search(r"\d+(k_\w+?)I", start.group(1))
            body = bodies.setdefault(start.group(1), []) if name and name.group(1) in KERNELS[src] else None
        elif text.startswith(".size"):
            body = None
        elif body is not None and text and not text.startswith(".") and not text.endswith(":"):
            body.append((text, inline))
    assert bodies and all(("s_barrier", True) in b for b in bodies.values())
    return bodies


def test_a_barrier_that_waits_for_loads_waits_for_lds_reads_too(functions):
    for name, body in functions.items():
        waits = [a for (a, _), b in zip(body, body[1:]) if b == ("s_barrier", True) and a.startswith("s_waitcnt") and "vmcnt" in a]
        assert waits and all("lgkmcnt(0)" in w for w in waits), (name, waits)


def test_no_lds_read_is_outstanding_at_a_barrier(functions):
    """In the order of the listing: a wait for all LDS operations between the last LDS read and any barrier."""
    for name, body in functions.items():
        pending = None
        for text, _ in body:
            if text.startswith("ds_read"):
                pending = text
            elif text.startswith("s_waitcnt") and "lgkmcnt(0)" in text:
                pending = None
            assert not (text == "s_barrier" and pending), (name, pending)


def test_kernels_without_a_mask_spill_nothing(functions):
    """A lane's sums take most of its registers: no value of the kernels without dropout lies in scratch memory."""
    plain = {n: b for n, b in functions.items()
             if re.search(r"k_adapter_(down_tilesILi\d+E|gemmILi\d+ELb[01]ELb[01]E|gemm_smallILi\d+ELb[01]ELb[01]E)Lb0E", n)}
    assert plain
    for name, body in plain.items():
        assert not [text for text, _ in body if text.startswith(("scratch_", "buffer_store_dword off"))], name
