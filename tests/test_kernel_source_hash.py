"""The recorded traffic figures belong to the attention kernel's code as it is."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "fp8_paged_kv_decode_gb300", "csrc")


def included(name):
    """The kernel directory's files that `name` includes, itself first."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    out = [name]
    for inc in re.findall(r'^#include "([^"]+)"', text, re.M):
        if os.path.exists(os.path.join(CSRC, inc)) and "/" not in inc:
            out += [x for x in included(inc) if x not in out]
    return out


def test_every_included_file_counts():
    files = included("decode_attn.cu")
    assert set(files) == set(bench.KERNEL_SOURCES) and "fp4_row.cuh" in files
    text = {}
    for f in files:
        with open(os.path.join(CSRC, f)) as fh:
            text[f] = fh.read()
    here = bench.kernel_source_hash()
    assert bench.kernel_source_hash(text) == here
    for f in files:
        assert bench.kernel_source_hash(dict(text, **{f: text[f] + "\n// a comment\n"})) == here
        assert bench.kernel_source_hash(dict(text, **{f: text[f] + "\nint x;\n"})) != here
