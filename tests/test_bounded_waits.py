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


def test_every_wait_is_one_of_the_helpers_that_the_selftest_runs():
    """A barrier is tested in helpers that give up by the clock, nowhere else, and fkv_selftest_wait runs each of them."""
    helpers = set()
    for name, text in SOURCES.items():
        for body in re.sub(r"//.*", "", text).split("\n}\n"):          # a function each (or several declarations)
            if not re.search(r"(?<!bool )\bmbar_try_wait(_sleep)?\(", body):
                continue
            head = re.findall(r"\n__device__ __forceinline__ bool (\w+)\(", body)
            assert len(head) == 1 and "globaltimer_ns()" in body, (name, head)
            helpers.add(head[0])
    assert helpers == {"mbar_wait_bounded", "mbar_wait_bounded_sleep", "tree_wait"}
    for h in helpers:
        assert h + "(bar" in SOURCES["selftest.cu"], h
