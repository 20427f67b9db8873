"""The serving example as its user runs it: prompts in chunks, then tokens one
by one, over gated maps on the exact path, against the same layers in float64.

Tolerance: every projection, attention and activation rounds its operands to
bf16 once (2^-8 of a value at most, in random directions ~2^-9.6 of a norm);
a layer has about eight such roundings on its way to the residual, and two
layers sixteen: sqrt(16) 2^-9.6 = 5e-3 of a block's output, which is less than
the residual.  2e-2 holds that with a margin of four.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layer.py")


@pytest.mark.parametrize("args", [
    ["--width", "512", "--heads", "8", "--kv-heads", "2", "--hidden", "1024", "--rank", "64", "--prompts", "70", "1", "333",
     "--chunk", "128", "--steps", "5"],
    ["--width", "1024", "--heads", "4", "--rank", "64", "--hidden", "2048", "--prompts", "200", "--chunk", "64", "--steps", "3"]])
def test_served_stack_matches_float64(args):
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("serve_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(args + ["--eps", "0", "--check"]) < 2e-2
