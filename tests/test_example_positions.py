"""The serving example makes its rotation table as long as the run can get (no GPU needed)."""
import importlib.util
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Made(Exception):
    pass


@pytest.mark.parametrize("steps", [1, 64, 1000, 20000])
def test_every_position_of_a_run_is_in_the_table(monkeypatch, steps):
    spec = importlib.util.spec_from_file_location("cached_decode", os.path.join(ROOT, "examples", "cached_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    made = {"max_pos": 4096}

    def model(**kw):
        made.update(kw)
        raise Made

    monkeypatch.setattr(mod, "Model", model)
    monkeypatch.setattr(sys, "argv", ["cached_decode.py", "--steps", str(steps)])
    with pytest.raises(Made):
        mod.main()
    # a warm-up step and `steps` more accept up to K + 1 = 8 tokens each; the last block lies behind all of the others
    assert made["max_pos"] >= 8 * (steps + 1)
