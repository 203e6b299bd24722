"""The binding's call extension (_calls.so) where it cannot be loaded: the
wrappers marshal in Python, and say so once."""

import os
import shutil

import pytest

import weight_only_int4_quantize_amd as awq


@pytest.fixture
def fresh(monkeypatch, tmp_path):
    awq.load()
    monkeypatch.setattr(awq, "_fast", None)
    monkeypatch.setattr(awq, "HERE", str(tmp_path))
    return tmp_path


def test_extension_not_built(fresh):
    ext, *entries = awq._fast_calls()
    assert ext is None and all(entries) and len(entries) == 4


@pytest.mark.parametrize("content", [b"", b"not an object file", "library"])
def test_extension_of_another_build(fresh, content):
    """An empty file, text, a library without the module's entry: what an
    interrupted or foreign build leaves."""
    path = os.path.join(fresh, "_calls.so")
    if content == "library":
        shutil.copy(awq.LIB_PATH, path)
    else:
        with open(path, "wb") as f:
            f.write(content)
    with pytest.warns(RuntimeWarning, match="_calls.so"):
        ext, *entries = awq._fast_calls()
    assert ext is None and all(entries) and len(entries) == 4
    assert awq._fast is not None        # decided once
