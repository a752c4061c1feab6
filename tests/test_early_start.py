"""Kernels that may start while the launch before them drains (programmatic dependent launch) read
their inputs coherently: the non-coherent load assumes data that stays the same for the whole
kernel, the time before its wait included, and a compiler may move it there."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_159_gb300", "csrc")


def _sources():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            yield os.path.basename(path), re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_non_coherent_load_behind_an_early_start():
    early = {n: t for n, t in _sources() if "griddepcontrol.wait" in t}
    assert "decode_int4.cuh" in early
    for name, text in early.items():
        assert not re.findall(r"__ldg\s*\(|ld\.global\.nc", text), name
        # and every kernel of the file waits before it does anything else
        assert text.count("pdl_wait();") == len(re.findall(r"__global__ void", text)), name


def test_every_early_start_is_of_a_kernel_that_waits():
    for name, text in _sources():
        if "cudaLaunchAttributeProgrammaticStreamSerialization" in text:
            assert "griddepcontrol.wait" in text, name
