"""The operators together, as examples/transformer_block.py runs them."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from conftest import ROOT


def example():
    spec = importlib.util.spec_from_file_location(
        "transformer_block", os.path.join(ROOT, "examples", "transformer_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.gpu
@pytest.mark.parametrize("args", [
    "--width 256 --heads 4 --kv-heads 2 --hidden 512 --lengths 100,0,33,1,200 --tune",
    "--width 1152 --heads 16 --kv-heads 16 --hidden 4608 --lengths 256 --full"])
def test_block(args):
    """Every operator against torch on the inputs it had: outputs are rounded to
    bf16 once (2^-8 of each element at most), attention's weights once more (2^-8 of
    each term), everything else is fp32."""
    from w4a4_mxfp4_activation_gb300 import build
    build.build()
    result = example().main(args.split())
    for name, off in result["off"].items():
        assert off < 2.0 ** -7, name
    assert result["cost"] < 1.0                       # closer to the exact block than nothing is
    if "before" in result:
        assert result["after"] < result["before"]


def test_example_refuses_widths_it_cannot_quantize():
    with pytest.raises(SystemExit):
        example().main(["--width", "100", "--heads", "4"])
