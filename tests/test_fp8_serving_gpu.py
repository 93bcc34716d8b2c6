"""The serving example runs its three operators together, eagerly and from a graph.

An e4m3 value is off by at most 2^-4 of itself, as a random rounding about 2^-4 / sqrt(3) = 0.036 of
its size.  A product of two such operands is then off by about 0.051 of its own size; the layer
behind it meets that error and two more quantised weights in a chain of three products: 0.051 +
0.036 x 3 = 0.16 at most, if the parts added up."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "fp8_serving.py")


@pytest.mark.parametrize("args", [[], ["--tokens", "1", "--d-model", "384", "--experts", "16"],
                                  ["--tokens", "33", "--d-model", "520", "--d-ff", "200"]])
def test_example(args):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("fp8_serving", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    projection, layer = example.main(args)
    assert projection <= 0.051 and layer <= 0.16
