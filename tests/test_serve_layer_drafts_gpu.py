"""The serving example with trees of drafts: the kept paths' rows against the layer in plain fp32."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("drafts", [7, 40])
def test_layer_with_drafts_follows_the_plain_one(drafts):
    spec = importlib.util.spec_from_file_location("serve_layer", os.path.join(ROOT, "examples", "serve_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # Keys and values to e4m3: each off by at most 2^-4 of itself, and a code shifted to a larger scale as the path moves
    # together by as much again.  Values enter the attention's output as a weighted mean; normed queries and keys of 64 dims
    # have scores of about 1 and never above 8 * 1.5^2, which move by about 2^-4 / sqrt(64) of that.  The output is one of three
    # terms of the layer's result: 0.1 of the result's norm bounds it, with the bf16 roundings (2^-8 each) well below.
    assert m.main(["--steps", "12", "--drafts", str(drafts), "--check"]) < 0.1
