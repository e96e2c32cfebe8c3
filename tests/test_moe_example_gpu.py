"""The example layer runs the operators together, checks itself against 64
bits and gives the same bits captured as eager."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")


@pytest.mark.parametrize("args", [[], ["--tokens", "1", "--experts", "16"],
                                  ["--tokens", "13", "--hidden", "520", "--inner", "264", "--experts", "9", "--topk", "3",
                                   "--rank", "12"]])
def test_moe_layer_example(args, capsys):
    spec = importlib.util.spec_from_file_location("moe_layer_example", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main(args + ["--replays", "3"])
    assert "one captured step" in capsys.readouterr().out
