"""Loading a library that does not fit the binding says to rebuild it (no GPU)."""
import subprocess

import pytest

import moe_expert_layer_topk_gb300 as m
from moe_expert_layer_topk_gb300 import build as b


def library(tmp_path, source):
    src, so = tmp_path / "old.c", tmp_path / "libold.so"
    src.write_text(source)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    return so


@pytest.mark.parametrize("source", [
    "int moe_abi_version(void) { return %d; }" % m.ABI_VERSION,      # of this version, before calls were added
    "int moe_abi_version(void) { return %d; }" % (m.ABI_VERSION - 1),
    "int something_else(void) { return 0; }",
])
def test_old_library_is_refused(tmp_path, source):
    b.build()
    good = m.lib()
    with pytest.raises(RuntimeError, match="rebuild"):
        m.lib(library(tmp_path, source))
    assert m.lib() is good
