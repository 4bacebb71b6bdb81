"""Dynamic shared memory starts where its declaration says: an array that a kernel
reads or writes 16 bytes at a time says 16, or the kernel rounds its address up."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "latent_projection_top_gb300", "csrc")
DECLARED = re.compile(r"extern __shared__\s+(?:__align__\((\d+)\)\s+)?(\w+)\s+(\w+)\[\];")
NATURAL = {"uint4": 16, "int4": 16, "float4": 16}


def arrays():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = open(path).read()
        found = list(DECLARED.finditer(text))
        assert len(found) == text.count("extern __shared__"), path
        for m, after in zip(found, found[1:] + [None]):
            body = text[m.end():after.start() if after else len(text)]
            yield pytest.param(m, body, id=f"{os.path.basename(path)}:{text[:m.start()].count(chr(10)) + 1}")


@pytest.mark.parametrize("declared,body", list(arrays()))
def test_dynamic_shared_memory_is_aligned(declared, body):
    align, kind, name = declared.groups()
    if int(align or NATURAL.get(kind, 1)) >= 16:
        return
    raw = re.search(rf"uint32_t (\w+) = ptx::smem_addr\({name}\);", body)
    assert raw, f"{kind} {name}[] is declared on less than 16 bytes, and used as it is"
    assert re.search(rf"\({raw[1]} \+ 1023u\) & ~1023u", body), f"{name}'s address is not rounded up"
