"""The serving example's rules: masks that would leave nothing to say, or are not of the vocabulary, are refused (CPU)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("allowed", [torch.zeros(100, dtype=torch.bool), torch.ones(99, dtype=torch.bool), torch.ones((1, 100), dtype=torch.bool),
                                     torch.ones(100)])
def test_masks_refused(allowed):
    spec = importlib.util.spec_from_file_location("serve_example", os.path.join(ROOT, "examples", "serve.py"))
    serve = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(serve)
    with pytest.raises(ValueError, match="allowed"):
        serve.Rules(allowed=allowed).tensors(2, 100, 10)
