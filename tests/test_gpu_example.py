"""The example that runs the decoder-layer operators together, at a small size."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_mlp.py")


@pytest.mark.parametrize("sizes", [(256, 640, 70, 5), (1040, 2048, 33, 16)])
def test_decoder_mlp(capsys, sizes):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("decoder_mlp", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    hidden, ffn, prompt, batch = sizes
    example.main([f"--hidden={hidden}", f"--ffn={ffn}", f"--prompt={prompt}", f"--batch={batch}", "--steps=3"])
    out = capsys.readouterr().out
    assert out.count("off by") == 4, out
