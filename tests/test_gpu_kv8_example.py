"""The serving example with rotary positions and an 8-bit cache runs, and its pages add up."""
import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_example_runs():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("attention_serving",
                                                  os.path.join(ROOT, "examples", "attention_serving.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    lens, samples, steps, turns = (200, 57), 3, 5, (33, 70)
    r = ex.serve8(lens, samples, steps, turns)
    assert r["prompt_out"].shape == (257, ex.HIDDEN) and r["turn_out"].shape == (103, ex.HIDDEN)
    for x in (r["prompt_out"], r["turn_out"], *r["outs"]):
        assert x.isfinite().all()
    pages = [(-(-n // 16), n // 16) for n in lens]
    own = [-(-(n + steps) // 16) - n // 16 for n in lens]
    assert r["before"] == sum(p for p, _ in pages) + samples * sum(own)
    assert r["live"] == sum(p for p, _ in pages)
    assert r["left"] == 256 - r["live"] - samples * sum(1 for n in lens if n % 16)
    # the second turns' pages follow
    assert int((r["cache"].refs > 0).sum()) == sum(-(-(n + t) // 16) for n, t in zip(lens, turns))
