"""The log-prob gap command's lines, each with the trainer that it is measured against."""
import pytest

from nvfp4_w4a4_moe_quant_amd import logprob_gap

pytestmark = pytest.mark.gpu
from gpu_util import say


def test_lines_name_their_trainer(monkeypatch, capsys):
    say("log-prob gap command")
    monkeypatch.setattr("sys.argv", ["logprob_gap", "2"])
    logprob_gap.main()
    lines = [t for t in capsys.readouterr().out.splitlines() if "log-prob gap|" in t]
    assert len(lines) == 4
    for t in lines:
        assert t.endswith("trainer on plain weights" if t.startswith("INT8 W8A8") else
                          "trainer on fake-quantized weights")
