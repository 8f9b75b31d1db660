"""The native part of the binding is checked against the release of torch it was built against: builds of that release
under another label (nightly, vendor, release candidate) are the same release, another number is not."""
import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def w8():
    __graft_entry__.build()
    import w8a8_int8_gemm_b200 as mod
    return mod


@pytest.mark.parametrize("label", ["", "+cu128", ".dev20260101+cu128", "a0+git1234567", "a0+0a1b2c3.nv25.12", "rc1",
                                   "rc3+cu129", ".post1"])
def test_builds_of_the_same_release(w8, label, monkeypatch):
    monkeypatch.setattr(torch, "__version__", w8._calls.torch_version + label)
    assert w8._load_calls() is w8._calls


@pytest.mark.parametrize("version", ["2.1.0", "1.13.1+cu117", "unknown", "", "{}1", "1{}"])
def test_other_releases(w8, version, monkeypatch):
    version = version.format(w8._calls.torch_version)
    monkeypatch.setattr(torch, "__version__", version)
    with pytest.raises(ImportError, match="was built against torch"):
        w8._load_calls()
