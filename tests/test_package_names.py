"""The package's names are those of its modules, at any time."""
import zero_sharded_mixed_gb300 as zero


def test_a_replaced_call_is_the_one_that_runs(zlib, monkeypatch):
    """A call replaced in the binding (a tracer around it, a stand-in) is reached by the
    package's name too, also where that name was used before, and so is the original
    once it is back."""
    for name in ("zero_linear", "zero_layout", "ZeroDropout"):
        original = getattr(zlib, name)
        assert getattr(zero, name) is original
        stand_in = lambda *a, **k: None  # noqa: E731
        with monkeypatch.context() as m:
            m.setattr(zlib, name, stand_in)
            assert getattr(zero, name) is stand_in
        assert getattr(zero, name) is original
