"""The Muon optimizer in the configuration, and how its step shares out the flat vector (CPU)."""
import pytest

from zero_sharded_mixed_gb300 import step as zs
from zero_sharded_mixed_gb300.config import ZeroConfig


def _cfg(params=None, **kw):
    return {"optimizer": {"type": "Muon", "params": params or {}}, **kw}


def test_muon_is_read():
    cfg = ZeroConfig.from_dict(_cfg({"lr": 0.01, "momentum": 0.9, "nesterov": False, "ns_steps": 7, "weight_decay": 0.1, "betas": [0.8, 0.9]}))
    assert (cfg.optimizer, cfg.lr, cfg.momentum, cfg.nesterov, cfg.ns_steps, cfg.weight_decay) == ("muon", 0.01, 0.9, False, 7, 0.1)
    assert cfg.betas == (0.8, 0.9)
    cfg = ZeroConfig.from_dict(_cfg())
    assert (cfg.momentum, cfg.nesterov, cfg.ns_steps) == (0.95, True, 5)
    assert ZeroConfig.from_dict({}).optimizer == "adamw"


@pytest.mark.parametrize("bad", [
    _cfg(zero_optimization={"stage": 3}), _cfg(gradient_clipping=1.0), _cfg(zero_optimization={"stage": 2, "zero_quantized_gradients": True}),
    _cfg({"momentum": 1.0}), _cfg({"momentum": -0.1}), _cfg({"ns_steps": 0}), _cfg({"ns_steps": 101}),
    {"optimizer": {"type": "Lion", "params": {}}},
])
def test_refusals(bad):
    with pytest.raises(ValueError):
        ZeroConfig.from_dict(bad)


def test_runs_of_touching_ranges():
    assert zs._runs([(0, 5), (5, 9), (12, 12), (12, 14), (20, 21)]) == [(0, 9), (12, 14), (20, 21)]
    assert zs._runs([]) == []


def test_equal_matrices_at_equal_distances_share_a_call():
    assert zs._batches([0, 100, 200, 300], 60, 10) == [(0, 4, 100)]
    assert zs._batches([0, 100, 200, 300], 60, 3) == [(0, 3, 100), (300, 1, 60)]
    assert zs._batches([0, 100, 250], 60, 10) == [(0, 2, 100), (250, 1, 60)]
    assert zs._batches([7], 60, 10) == [(7, 1, 60)]
    assert zs._batches([0, 60, 120], 60, 1) == [(0, 1, 60), (60, 1, 60), (120, 1, 60)]
