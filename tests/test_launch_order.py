"""Reading of the attention gradients' launchers (no GPU): nothing is on the
stream before every check has passed.

A call that is refused must leave the caller's workspace untouched, so that it
may be freed or used on another stream at once.  From a launcher's first kernel
on, its code holds no refusal, no tensor map, no kernel attribute and no other
launcher that could refuse."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_block_self_b200", "csrc")
REFUSALS = r"NLE_ERR_(INVALID_ARG|UNSUPPORTED|MISALIGNED)|encode_tmap|allow_max_dynamic_smem|\blaunch_\w+\("


def _body(path, name):
    src = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(os.path.join(CSRC, path)).read(), flags=re.S)
    m = re.search(rf"\bint {name}\([^)]*\)\s*\{{", src)
    depth, i = 1, m.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        i += 1
    return src[m.end():i]


@pytest.mark.parametrize("path,name", [("attn_bwd_sm100a.cu", "launch_attn_bwd"),
                                       ("block_bwd_sm100a.cu", "launch_block_bwd")])
def test_no_refusal_behind_the_first_kernel(path, name):
    body = _body(path, name)
    first = re.search(r"<<<|\blaunch_attn_delta\(", body)
    late = re.search(REFUSALS, body[first.end():])
    assert late is None, f"{path}, {name}: {late.group()} behind the first kernel"
