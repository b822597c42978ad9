"""A time-out that a kernel reports names its wait by a number: no two source files share one, so that it also names the kernel."""
import glob
import os
import re

from hybrid_upcycling_gb300 import build


def test_numbers_of_waits_name_one_source_file():
    files = {}
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        text = open(path).read()
        sites = re.findall(r"\bctl,\s*(\d+)\)", text) + re.findall(r"kDevTimeoutBase \+ (\d+)", text)
        calls = len(re.findall(r"\b(?:wait_bounded|wait_count)(?:<true>)?\(", text)) - len(re.findall(r"bool wait_(?:bounded|count)\(", text))
        assert len(sites) >= calls or "int site" in text, path  # every wait was recognised
        for s in set(map(int, sites)):
            files.setdefault(s, []).append(os.path.basename(path))
    assert len(files) > 30
    assert {s: f for s, f in files.items() if len(f) > 1} == {}
