"""The serving example: the three calls with tl_gemm as one decoder layer, against the layer in plain fp32."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layer_follows_the_plain_one():
    spec = importlib.util.spec_from_file_location("serve_layer", os.path.join(ROOT, "examples", "serve_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # Keys and values to e4m3: each off by at most 2^-4 of itself.  Values enter the attention's output as a weighted
    # mean (2^-4 at most, far less for many keys); scores of a few units move by about 2^-4 / sqrt(64) of |q||k| / 8.
    # The output is one of three terms of the layer's result (x itself, attention, experts): 0.1 of the result's norm
    # bounds it, with the bf16 roundings of the intermediate tensors (2^-8 each) well below.
    assert m.main(["--steps", "20", "--check"]) < 0.1
