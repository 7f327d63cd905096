"""What the built library's kernels take, from the code objects' own notes, without a GPU."""
import os
import re
import subprocess

import pytest

READELF = "/opt/rocm/llvm/bin/llvm-readelf"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: [(offset, size, kind) of each argument]} of libsvd.so."""
    import lossless_draft_verification_verifier_amd as svd
    data = open(svd.LIB_PATH, "rb").read()
    out, at = {}, data.find(b"\x7fELF", 4)
    path = str(tmp_path_factory.mktemp("code") / "object")
    while at >= 0:
        with open(path, "wb") as f:
            f.write(data[at:])
        notes = subprocess.run([READELF, "--notes", path], capture_output=True, text=True).stdout
        for k in re.split(r"\n  - (?=\.)", notes):
            name = re.search(r"\.name: +(\S*kr_\w+)", k)
            if name:
                args = re.findall(r"\.offset: +(\d+)\s+\.size: +(\d+)\s+\.value_kind: +(\w+)", k)
                out[name.group(1)] = [(int(o), int(s), kind) for o, s, kind in args]
        at = data.find(b"\x7fELF", at + 4)
    assert len(out) > 100, "the notes were not read"
    return out


def test_arguments_read_again_begin_the_arguments(kernels):
    # kr_tree_attention reads its arguments a second time, by the address at which they begin:
    # one parameter of its own, at offset 0
    mine = {n: a for n, a in kernels.items() if "kr_tree_attention" in n}
    assert len(mine) == 48
    for n, args in mine.items():
        own = [a for a in args if not a[2].startswith("hidden_")]
        assert len(own) == 1 and own[0][0] == 0 and own[0][2] == "by_value", (n, own)
