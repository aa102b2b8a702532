"""The serving example: prompts, single tokens, forked samples and a compacted
pool together, against whole sequences."""

import importlib.util
import os

import pytest

from gpu_harness import gpu_or_skip

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_decoder.py")


@pytest.mark.parametrize("args", [
    "--layers 2 --steps 5",
    "--layers 1 --hidden 512 --heads 7 1 128 --prompts 17 33 1 700 --samples 3 --steps 3 --page 32",
    "--layers 1 --hidden 256 --heads 4 4 64 --prompts 64 --samples 0 --steps 2 --page 64",
])
def test_served_steps_equal_whole_sequences(args):
    gpu_or_skip()
    spec = importlib.util.spec_from_file_location("serve_decoder", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    print("example", args, flush=True)
    # per layer: bf16 roundings of the residual stream (2), attention's p and output (2), the linears' outputs (4) and
    # the norms (2), each off by at most 2^-8 relative and differently on the two paths: far below this
    assert example.main(args.split()) < 2e-2
