"""Kernels that may be resident before the launch before them has ended (`launch_after`) wait for it
first, and declare none of what it writes as memory that does not change: `const __restrict__` would
let the compiler read it through the non-coherent path, and ahead of that wait."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_kv_cache_kv4_b200", "csrc")


def sources():
    return {f: open(os.path.join(CSRC, f)).read() for f in sorted(os.listdir(CSRC))}


def early_kernels():
    """(file, signature, body) of every kernel that launch_after launches."""
    src = sources()
    names = {n for s in src.values() for n in re.findall(r"launch_after\((\w+)[<,]", s)}
    out = []
    for f, s in src.items():
        for n in names:
            at = re.search(r"__global__[^;{]*\b%s\(" % n, s)
            if at:
                body = s.index("{", at.end())
                out.append((f, s[at.end():body], s[body:s.index("\n}\n", body)]))
    assert len(out) == len(names) == 2
    return out


def test_they_wait_before_they_read():
    for f, _, body in early_kernels():
        wait = body.index("wait_for_launch_before();")
        for read in ("notes", "partials"):
            assert body.index(read) > wait, f


def test_nothing_they_read_is_declared_constant():
    for f, signature, body in early_kernels():
        assert "__restrict__" not in signature, f
        assert "__ldg(" not in body, f
        assert not re.search(r"= notes\[", body), f  # (through L2, as the records: read_note)
