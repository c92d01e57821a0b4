"""Each call's first kernel reads its inputs behind its grid wait: the kernel
before it on the stream may have let it start before it wrote them, and what
it writes is only promised to be visible behind the wait.  Read from the
sources, since a race need not show when it runs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "precision_moe_grouped_gb300", "csrc")

# kernel, and what names its inputs in its body
FIRST = [("route.cu", "route_kernel", ("logits",)),
         ("route.cu", "route_expand_tiny_kernel", ("logits", "quantize_token")),
         ("adapters.cu", "group_kernel", ("ids[",)),
         ("adapters.cu", "small_kernel", ("tiles.find", "blocks.fetch", "row[j]")),
         ("balance.cu", "balance_count_kernel", ("ids +", "mask[")),
         ("balance.cu", "balance_small_kernel", ("rows.load", "a.ids", "is_on(t)")),
         ("adamw.cu", "adamw_kernel", ("take_block", "grad_scale"))]


def braces(text, at):
    """The block that begins at text[at] == "{"."""
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError("unbalanced")


def body(source, name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    at = re.search(r"__global__[^;{]*\b%s\(" % name, text).end()
    return braces(text, text.index("{", at))


@pytest.mark.parametrize("source,name,inputs", FIRST, ids=[f[1] for f in FIRST])
def test_inputs_are_read_behind_the_wait(source, name, inputs):
    text = body(source, name)
    if name == "route_expand_tiny_kernel":   # CTAs that only prefetch: a wrong guess costs time alone
        guess = braces(text, text.index("{", text.index("if (t >= T)")))
        assert "griddep" not in guess and "bulk_prefetch_l2" in guess and "ids[" not in guess
        text = text.replace(guess, "")
    ahead = text[:text.index("griddep_wait()")]
    assert text.count("griddep_wait()") == 1
    for word in inputs:
        assert word in text and word not in ahead, (name, word)
