"""The bf16 products and the adapters keep their registers: no compiled kernel of theirs uses scratch memory."""

import os
import re
import shutil
import subprocess

import pytest

import fp4_grouped_gemm_amd as fgg
from test_wait_states import code_objects

READELF = shutil.which("llvm-readelf") or "/opt/rocm/llvm/bin/llvm-readelf"

pytestmark = [pytest.mark.skipif(not os.path.exists(fgg.library_path()),
                                 reason="libfgg.so not built (run __graft_entry__.build())"),
              pytest.mark.skipif(not os.path.exists(READELF), reason="no llvm-readelf")]


def test_products_and_adapters(tmp_path):
    sizes = {}
    for i, o in enumerate(code_objects(fgg.library_path())):
        f = tmp_path / f"{i}.co"
        f.write_bytes(o)
        notes = subprocess.run([READELF, "--notes", str(f)], capture_output=True, text=True, check=True).stdout
        names = re.findall(r"^ +\.name: +(_Z\S+)$", notes, re.M)
        scratch = re.findall(r"^ +\.private_segment_fixed_size: +(\d+)$", notes, re.M)
        assert len(names) == len(scratch)
        sizes.update(zip(names, map(int, scratch)))
    ours = {n: s for n, s in sizes.items() if re.search("gemm_bf16_kernel|rows_bf16_kernel|dw_join_kernel|lora_", n)}
    assert len(ours) == 15 + 2 + 4 + 27
    assert not any(ours.values()), {n: s for n, s in ours.items() if s}
