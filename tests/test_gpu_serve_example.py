"""The serving example: its decoding gives the logits that the same sequences give as prompts."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args", [["--tokens", "12"], ["--no-graph", "--batch", "3", "--prompt", "70", "--tokens", "5"],
                                  ["--layers", "8", "--batch", "1", "--tokens", "20"]])
def test_example(args):
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location("serve_hybrid", os.path.join(ROOT, "examples", "serve_hybrid.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # Eight bf16 roundings a layer (2^-9 rms relative each, at worst adding up) on either side, eight layers:
    # sqrt(8 * 8 * 2) 2^-9 = 2.2e-2 where the errors are independent, and twice that for what the layers amplify.
    assert example.main(args) <= 5e-2
