"""What the attention kernels write and the merge reads, the merge being resident
before they end, is not read through the non-coherent path: __ldg is for what no
kernel of a call writes."""
import os
import re

from exact_attention_forward_tiled_gb300 import build as fa_build


def test_read_only_loads():
    seen = 0
    for name in sorted(os.listdir(fa_build.CSRC)):
        if not name.startswith("kv_"):
            continue
        text = re.sub(r"//[^\n]*", "", open(os.path.join(fa_build.CSRC, name)).read())
        for m in re.finditer(r"__ldg\(", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            arg = text[m.end():end - 1]
            seen += 1
            assert not re.search(r"\bcum\b|part_o|part_ml|\.ml\b|(own|pre)\.o\b", arg), f"{name}: __ldg({arg})"
    assert seen > 5
