"""What the kernels do when a wait gives up, as far as their source shows it without a GPU."""
import os
import re

from fp8_paged_kv_decode_gb300 import _build

SOURCES = {f: open(os.path.join(_build.CSRC, f)).read() for f in sorted(os.listdir(_build.CSRC)) if f.endswith((".cu", ".cuh"))}
VOTE = re.compile(r"__any_sync\(kAll,|group_any\(\d|both_any\(")


def test_threads_leave_together():
    """Warps meet at barriers without a limit: whether a thread leaves its loop because a wait has given up is decided by a
    vote of all that it meets there, not by itself."""
    seen = 0
    for name, text in SOURCES.items():
        for line in text.splitlines():
            code = line.split("//")[0]
            if "*dead" not in code or not re.search(r"\b(break|while|for)\b", code):
                continue
            seen += 1
            vote = VOTE.search(code)
            assert vote and vote.start() < code.index("*dead"), (name, line)
    assert seen >= 8
