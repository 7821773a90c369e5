"""A checkpoint says whose moments it holds, and an engine of the other optimizer refuses it."""
import json
import os

import pytest
import torch

from zero_sharded_mixed_gb300 import binding as zb
from zero_sharded_mixed_gb300 import checkpoint as ck
from zero_sharded_mixed_gb300.config import ZeroConfig
from zero_sharded_mixed_gb300.engine import ZeroEngine

NUMELS = [48, 7]


def _state(L):
    return [torch.arange(L.padded_n, dtype=torch.float32) + i for i in range(3)]


def _save(path, L, **kw):
    return ck.save(path, L, NUMELS, *_state(L), 3, zb.ZeroAdamW.make(step=3), **kw)


def test_the_name_is_kept_and_checked(tmp_path):
    L = zb.zero_layout(NUMELS, 2)
    for kw, name, other in (({}, "adamw", "muon"), ({"optimizer": "muon"}, "muon", "adamw")):
        path = tmp_path / name
        _save(path, L, **kw)
        assert ck.load_meta(path)["optimizer"] == name
        got = [torch.zeros(L.padded_n) for _ in range(3)]
        with pytest.raises(ValueError, match=name):
            ck.restore(path, L, *got, optimizer=other)
        assert all(int(t.count_nonzero()) == 0 for t in got)
        for want in (name, None):
            assert ck.restore(path, L, *got, optimizer=want) == 3
            assert all(torch.equal(a, b) for a, b in zip(got, _state(L)))
        ck.reshard(path, tmp_path / f"{name}_3", 3)
        assert ck.load_meta(tmp_path / f"{name}_3")["optimizer"] == name
        assert ck.consolidate(path)["step"] == 3


def test_a_checkpoint_without_a_name_goes_with_any(tmp_path):
    """As those written before there was one, of either optimizer; resharded it has none still."""
    L = zb.zero_layout(NUMELS, 2)
    _save(tmp_path, L)
    path = os.path.join(tmp_path, ck.META)
    with open(path) as f:
        meta = json.load(f)
    del meta["optimizer"]
    with open(path, "w") as f:
        json.dump(meta, f)
    got = [torch.zeros(L.padded_n) for _ in range(3)]
    for name in ("adamw", "muon", None):
        assert ck.restore(tmp_path, L, *got, optimizer=name) == 3
    ck.reshard(tmp_path, tmp_path / "3", 3)
    assert ck.load_meta(tmp_path / "3").get("optimizer") is None


@pytest.mark.gpu
@pytest.mark.parametrize("stage", [1, 2])
def test_engines(zlib, cuda_device, tmp_path, stage):
    def engine(kind):
        cfg = ZeroConfig.from_dict({"zero_optimization": {"stage": stage}, "optimizer": {"type": kind, "params": {"lr": 1e-2}}})
        return ZeroEngine(NUMELS, 2, cfg, shapes=[(6, 8), (7,)])

    engines = {}
    for kind in ("AdamW", "Muon"):
        e = engines[kind] = engine(kind)
        e.backward(torch.ones(2, e.L.padded_n, dtype=torch.bfloat16, device="cuda"))
        e.step()
        e.save_checkpoint(tmp_path / kind)
    for kind, other in (("AdamW", "Muon"), ("Muon", "AdamW")):
        e = engine(kind)
        with pytest.raises(ValueError):
            e.load_checkpoint(tmp_path / other)
        assert e.t == 0 and int(e.m.count_nonzero()) == 0
        assert e.load_checkpoint(tmp_path / kind) == 1
        assert torch.equal(e.m, engines[kind].m) and torch.equal(e.weights, engines[kind].weights)
