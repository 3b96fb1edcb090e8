"""The examples make the calls that they say they make."""
import glob
import os
import re

import pytest

import quantized_q4_weight_gb300 as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EXAMPLES = sorted(glob.glob(os.path.join(ROOT, "examples", "*.py")))


@pytest.mark.parametrize("path", EXAMPLES, ids=[os.path.basename(p) for p in EXAMPLES])
def test_calls_named_in_the_docstring_are_made(path):
    text = open(path).read()
    doc, code = text.split('"""', 2)[1:]
    named = {n for inside in re.findall(r"\(([a-z0-9_, ]+)\)", doc) for n in inside.replace(",", " ").split() if hasattr(q, n)}
    assert named and all(re.search(rf"\bq\.{n}\(", code) for n in named), sorted(n for n in named if f"q.{n}(" not in code)
