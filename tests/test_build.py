"""The build where the binding's compiler fails: the C library is built all the same, and what is missing says so when it is used."""
import os
import warnings

import pytest

from gated_delta_rule_34_gb300 import build, cache


@pytest.fixture(autouse=True)
def built():
    build.build()


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkda.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "binding.so"))
    return monkeypatch


def test_the_library_does_not_need_the_binding(elsewhere):
    elsewhere.setattr(build, "CXX", "false")
    with pytest.warns(RuntimeWarning, match="cache_binding"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    with pytest.raises(RuntimeError, match="build it with"):
        cache._binding.__wrapped__()


def test_no_such_compiler(elsewhere):
    elsewhere.setattr(build, "CXX", "/no/such/compiler")
    with pytest.warns(RuntimeWarning, match="/no/such/compiler"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_a_binding_of_other_sources_does_not_stay(elsewhere):
    with open(build.BINDING, "wb") as f:
        f.write(b"an older build's")
    os.utime(build.BINDING, (1, 1))
    elsewhere.setattr(build, "CXX", "false")
    with pytest.warns(RuntimeWarning):
        build.build()
    assert not os.path.exists(build.BINDING)


def test_a_good_build_says_nothing(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkda.so"))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
