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


def test_operator_times(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("operator_times", PATH.replace("decoder_mlp", "operator_times"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main(["q8_token", "--case=op=w4,M=3,N=80,K=264,zeros=True", "--case=op=norm_backward,rows=5,hidden=64"])
    lines = capsys.readouterr().out.splitlines()
    example.main(["q8_token", "--calls=2"])
    assert capsys.readouterr().out.splitlines() == ["q8_token"]
    assert [ln.split()[0] for ln in lines] == ["q8_token", "op=w4,M=3,N=80,K=264,zeros=True",
                                               "op=norm_backward,rows=5,hidden=64"]
    assert all("in a graph" in ln for ln in lines)
