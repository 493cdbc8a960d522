"""When the library and the extension module are built anew."""
import os

import pytest

import kv_cache_quantize_b200 as kvq
from kv_cache_quantize_b200 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_nothing_is_stale_after_a_build():
    assert not build.needs_build()


def test_another_torch_makes_the_extension_stale(monkeypatch):
    """The extension is built against the installed torch's headers: another version, or another Python, needs a new one."""
    monkeypatch.setattr(build, "installed_torch", lambda: "0.0.1 cpython-00")
    assert build.needs_build()


def test_an_extension_of_unknown_origin_is_stale(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "CALLS_TORCH", str(tmp_path / "none"))
    assert build.needs_build()


def test_an_extension_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    stamp = tmp_path / "stamp"
    stamp.write_text("0.0.1 cpython-00")
    monkeypatch.setattr(build, "CALLS_TORCH", str(stamp))
    monkeypatch.setattr(kvq, "_CALLS", None)
    with pytest.raises(RuntimeError, match="0.0.1"):
        kvq._calls()
    os.remove(stamp)                           # nothing known: it is tried
    assert kvq._calls().copy_pages
