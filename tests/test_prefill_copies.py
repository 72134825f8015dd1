"""Bulk copies of the prefill kernel: each role that starts some waits for them before it ends, on every way out, so that none
lands in shared memory that the CTA has given back.  Read in the source: the ways out that matter are a lost copy's."""
import os
import re

import query_aware_sparse_kv_gb300 as qskv

PATH = os.path.join(os.path.dirname(qskv.__file__), "csrc", "prefill_tc.cu")


def _roles():
    """(name, body) of every role of the kernel, comments left out."""
    text = re.sub(r"//[^\n]*", "", open(PATH).read())
    for m in re.finditer(r"__device__[^;{]*?\s(\w+_role)\s*\([^;{]*\)\s*\{", text):
        yield m.group(1), text[m.end():text.index("\n}", m.end())]


def test_a_role_waits_for_its_own_copies():
    roles = dict(_roles())
    assert set(roles) == {"softmax_role", "mma_role", "load_role", "fetch_role", "convert_role", "list_role"}
    copying = {name for name, body in roles.items() if re.search(r"\b(tma_load_\w+|bulk_load)\(", body)}
    assert copying == {"load_role", "fetch_role", "list_role"}
    for name in copying:
        body = roles[name]
        alias = dict(re.findall(r"uint64_t \*(\w+) = &s\.(\w+)", body))
        barriers = {alias.get(x, x) for x in re.findall(r"mbar_arrive_expect_tx\(&?(?:s\.)?(\w+)", body)}
        assert barriers
        last = max(m.end() for m in re.finditer(r"\b(tma_load_\w+|bulk_load)\(", body))
        # behind the loop (a statement of the function's own depth) that the copies are in
        end = body[last:].split("\n    }\n", 1)
        assert len(end) == 2, name
        waits = set(re.findall(r"mbar_wait_bounded\(&s\.(\w+)", end[1]))
        assert waits == barriers, (name, waits, barriers)
        loop = body[re.search(r"\n    (while|for) \(", body).start():]
        assert "return;" not in loop, name
