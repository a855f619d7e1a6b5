"""Kernels launched early (programmatic dependent launch) touch no global
memory before grid_dependency_wait(): read off the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_415_b200", "csrc")
# What reads or writes global memory in these kernels, by any route.
TOUCHES = re.compile(r"context_lens\[|query_starts\[|block_tables\[|slot_mapping\[|positions\[|"
                     r"checked_context\(|prompt_span\(|attend_size\(|tma_(load|store)|bulk_copy|"
                     r"status_or\(|ld_\w+\(|__ldg\(|ws_\w+\[|atomic")


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            name = re.search(r"(\w+)\s*\((?!\s*\d|\s*k[A-Z])", text[m.end():]).group(1)
            start = text.index("{", text.index(")\n{", m.end()))
            depth = 0
            for end in range(start, len(text)):
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                if depth == 0:
                    break
            yield pytest.param(text[start:end], id=f"{os.path.basename(path)}:{name}")


@pytest.mark.parametrize("body", list(_kernels()))
def test_no_global_access_before_the_wait(body):
    at = body.find("grid_dependency_wait();")
    if at < 0:
        # not launched early: it then must not let others begin early either
        assert "allow_dependents();" not in body
        return
    early = TOUCHES.search(body[:at])
    assert early is None, f"{early.group(0)} before the wait"
    assert "allow_dependents();" not in body[:at]
