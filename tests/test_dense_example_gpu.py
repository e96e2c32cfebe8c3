"""The example of a dense layer's projections runs, checks itself against 64
bits, its gradients too, and gives the same bits captured as eager."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "dense_layer.py")


@pytest.mark.parametrize("args", [[], ["--tokens", "1"], ["--tokens", "301", "--hidden", "520", "--inner", "264", "--heads", "7",
                                                          "--kv", "1", "--dim", "72"],
                                  ["--tokens", "13", "--hidden", "51", "--inner", "33", "--heads", "3", "--kv", "3", "--dim", "10"]])
def test_dense_layer_example(args, capsys):
    spec = importlib.util.spec_from_file_location("dense_layer_example", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    example.main(args + ["--replays", "3"])
    assert "one captured step" in capsys.readouterr().out
