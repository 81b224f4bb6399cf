"""bench.py reports a recorded traffic figure only for the sources it was measured on: the files it hashes for a kernel are
the one that holds the kernel and every header of the library that it includes, directly or not.  (The public header is
left out: it is all documentation and signatures but for a few limits.)"""
import re
import sys
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
sys.path.insert(0, str(ROOT))
import bench  # noqa: E402

CSRC = ROOT / "paged_kv_cache_275_gb300" / "csrc"


def included(path: Path) -> set[Path]:
    found, todo = set(), [path]
    while todo:
        p = todo.pop()
        if p in found or not p.exists():
            continue
        found.add(p)
        todo += [CSRC / name for name in re.findall(r'^\s*#include "([^"]+)"', p.read_text(), re.M)]
    return found


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_every_included_header_is_hashed(kernel):
    listed = [ROOT / rel for rel in bench.KERNEL_SOURCES[kernel]]
    assert re.search(rf"\b{kernel}\b", listed[0].read_text())
    assert set(listed) == included(listed[0])
