"""The serving example: its steps agree with attention over the whole sequence."""
import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_decoded_tokens_match_whole_sequences():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("attention_serving",
                                                  os.path.join(ROOT, "examples", "attention_serving.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    lens, samples, steps = (200, 57), 3, 5
    r = ex.serve(lens, samples, steps)
    layer, at = r["layer"], 0
    for i, n in enumerate(lens):
        for s in range(samples):
            # the sample's whole sequence at once, over the cache's FP16 keys and values
            x = torch.cat([r["prompts"][at:at + n]] + [t[i * samples + s][None] for t in r["tokens"]])
            q, k, v = layer.qkv(x)
            whole = layer.out(ex.cf.comp_attn_f32x16(q, k.half(), v.half()))
            for step in range(steps):
                got, want = r["outs"][step][i * samples + s], whole[n + step]
                # The two projections (other row counts, other kernels) differ by about 1e-7, so a
                # part of some 1e-7 / 2^-10 = 1e-4 of the FP16 keys and values rounds the other way,
                # by 2^-10 each: about 2^-10 sqrt(1e-4) = 1e-5 of the output from the values and as
                # much from the keys.  Ten times that; a wrong page or token changes about 0.1.
                assert float((got - want).norm() / want.norm()) < 1e-4
        at += n
    # 200 tokens: 13 pages, 57: 4; a fork shares the full ones and has its own from there on
    pages = [(-(-n // 16), n // 16) for n in lens]
    own = [-(-(n + steps) // 16) - n // 16 for n in lens]
    assert r["before"] == sum(p for p, _ in pages) + samples * sum(own)
    assert r["live"] == sum(p for p, _ in pages)
    table = r["cache"].table
    assert sorted(p for p in table.flatten().tolist() if p >= 0) == list(range(r["live"]))
