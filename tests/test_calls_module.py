"""The compiled module behind the paged and windowed calls."""

import os
import subprocess
import sys

import pytest


@pytest.fixture(scope="module")
def ub():
    from kv_cache_reuse_falcon_b200 import build
    build.build()
    from kv_cache_reuse_falcon_b200 import binding
    return binding


@pytest.mark.parametrize("name,count", [("pool_write", 14), ("decode", 19), ("evict", 14), ("prefill", 14),
                                        ("prefill_bwd", 19)])
def test_calls_check_the_number_of_their_arguments(ub, name, count):
    f = getattr(ub._calls, name)
    for n in (0, 1, count - 1, count + 1):
        with pytest.raises(TypeError, match="%d arguments by position, got %d" % (count, n)):
            f(*[None] * n)
    with pytest.raises(ValueError):          # the right number, of no tensors
        f(*[None] * count)


def test_the_module_belongs_to_one_torch(monkeypatch):
    """Its file is named after torch's version and Python's ABI: another torch finds it not built."""
    import sysconfig

    import torch
    from kv_cache_reuse_falcon_b200 import build
    build.build()
    mine = build.calls_path()
    assert os.path.exists(mine) and mine.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and build.up_to_date()
    monkeypatch.setattr(torch, "__version__", "9.8.7+other")
    assert build.calls_module() == "_calls_torch_9_8_7_other" and build.calls_path() != mine
    assert not build.up_to_date()


def test_other_calls_work_without_the_module():
    """Where it cannot be loaded, the calls through the library do, and a paged call says what is missing."""
    code = """if True:
        from kv_cache_reuse_falcon_b200 import build
        build.calls_module = lambda: "_calls_of_no_torch"
        from kv_cache_reuse_falcon_b200 import binding as ub
        assert ub.status_string(0) == "UNIPIN_OK" and ub.masked_prefill_workspace_size() == 256
        try:
            ub.paged_evict(None, None, None, 0, None, None, 1, 1)
        except ImportError as e:
            assert "_calls_of_no_torch" in str(e) and "build" in str(e)
        else:
            raise SystemExit("no error")
        """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root)
