"""The times of the layer operators' cases, at small sizes."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "operator_times.py")


def test_operator_times_of_the_layer(capsys):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("operator_times", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    cases = ["op=moe,T=5,E=8,H=264,I=72,top_k=2", "op=lora,M=90,N=130,K=264", "op=norm_backward,rows=5,hidden=64"]
    example.main(["--more", "norm_token"] + [f"--case={c}" for c in cases])
    lines = capsys.readouterr().out.splitlines()
    assert [ln.split()[0] for ln in lines] == ["norm_token"] + cases
    assert all("in a graph" in ln for ln in lines)
    with pytest.raises(SystemExit):
        example.main(["--more", "--case=op=q8,M=1,N=80,K=264"])
