"""Loads behind an early launch, by reading the sources. Every kernel lets its
successor start before it has ended (programmatic dependent launch), so what a
kernel reads may still be written while it is resident. griddepcontrol.wait
covers ordinary loads; the read-only path (__ldg, ld.global.nc, or a
__restrict__ pointer that lets the compiler choose it) wants data that nothing
writes for the kernel's whole life. No timing on a GPU can show that such a load
is sound, so the sources must not have one."""
import glob
import os
import re

from paged_kv_cache_60_gb300 import build as dabuild

SOURCES = sorted(glob.glob(os.path.join(dabuild.CSRC, "*.cu*")))


def _code(path):
    text = open(path).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_no_load_takes_the_read_only_path():
    assert len(SOURCES) >= 10
    found = [(os.path.basename(f), m.group(0)) for f in SOURCES
             for m in re.finditer(r"__ldg\b|\bld\.global\.nc\b|__restrict(__)?\b", _code(f))]
    assert not found, found


def test_every_kernel_waits_before_it_reads():
    """Each __global__ function waits for the grids before it, and lets the next start only then."""
    for f in SOURCES:
        code = _code(f)
        for body in re.split(r"__global__", code)[1:]:
            wait, go = body.find("pdl_wait()"), body.find("pdl_launch_dependents()")
            assert 0 <= wait < go, os.path.basename(f)
