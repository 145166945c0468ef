"""The speculative-decoding calls chained as a serving loop uses them (examples/speculative_step.py)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("kw", [dict(), dict(batch=1, prompt=17, steps=9, nodes=40, seed=1), dict(batch=7, nodes=1, seed=2)])
def test_the_kept_cache_is_the_plainly_appended_one(kw):
    path = os.path.join(ROOT, "examples", "speculative_step.py")
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    flags, same, length = mod.main(**kw)
    assert flags == 0 and same and min(length) > 0
