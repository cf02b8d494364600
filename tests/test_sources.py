"""What the library's sources may not contain."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_bf16_gemm_persistent_gb300", "csrc")


def test_no_load_with_cluster_multicast():
    """The library runs in every process of a job on several GPUs: no TMA load in it is multicast over a cluster.
    (The commit of a pair's MMAs, which signals barriers and moves no data, may be.)"""
    files = [f for pattern in ("*.cu", "*.cuh", "*.cpp", "*.h") for f in glob.glob(os.path.join(CSRC, pattern))]
    assert len(files) >= 8
    for path in files:
        with open(path) as f:
            for asm in re.findall(r'"[^"\n]*\.multicast[^"\n]*"', f.read()):
                assert "tcgen05.commit" in asm, (path, asm)


def test_no_non_coherent_load_in_kernels_that_start_early():
    """Kernels that are launched while the one before still runs (host.h: Launch) read what that one may be writing, and
    some write in the place of an input: ld.global.nc and __ldg are for memory that nobody writes as long as a kernel lives."""
    for name in ("layernorm.cuh", "lora_kernel.cuh", "moe_kernel.cuh", "rowwise.cuh", "skinny.cuh", "w4_kernel.cuh"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert "ld.global.nc" not in text and "__ldg" not in text, name
