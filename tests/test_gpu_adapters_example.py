"""The example that trains two adapters and serves them together: training
lowers the error, and the served batch is what each adapter gives alone (two
bf16 roundings, act and out, that may fall differently: under 2^-8 of the norm)."""
import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
def test_train_two_adapters_and_serve_them(cuda_available, fmt):
    from weight_quantized_swiglu_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("adapters_example", os.path.join(ROOT, "examples", "adapters.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    results, off = ex.main(["--fmt", fmt])
    for losses in results:
        assert losses[-1] < 0.25 * losses[0], losses
    assert off <= 2.0 ** -8
