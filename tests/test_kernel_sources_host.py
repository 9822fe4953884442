"""What the kernels' sources declare; no GPU."""
import glob
import os
import re

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "block_quantized_matmul_gq_gb300", "csrc", "*.cu*")))


def test_shared_arrays_are_aligned_for_vectors():
    """A dynamic shared array begins where its declaration's alignment allows. One that is read in words of 16 bytes
    says so, or (smem_raw) is aligned by its kernel."""
    seen = 0
    for path in SOURCES:
        text = open(path).read()
        for align, kind, name in re.findall(r"extern __shared__ (?:__align__\((\d+)\) )?(\w+) (\w+)\[\]", text):
            seen += 1
            if name == "smem_raw":
                assert re.search(r"(smem_addr\(smem_raw\)|raw_addr) \+ 1023u\) & ~1023u", text), path
            elif kind not in ("int", "float"):
                assert align and int(align) >= 16, f"{os.path.basename(path)}: {kind} {name}[]"
    assert seen >= 9
