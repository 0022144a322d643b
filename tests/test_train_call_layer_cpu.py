"""The extension that marshals the training operators' calls: the library and
the other calls do without it, and its file says what it was built for."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_WITHOUT = """
import torch
from dit_long_sequence_gb300 import build
build.calls_path = lambda: "/nowhere/dit_calls.so"
import dit_long_sequence_gb300 as dl
from dit_long_sequence_gb300 import binding
assert callable(dl.attn_fwd) and binding.raw().dit_version() > 0 and dl.rope_inv_freq(8)[0].numel() == 4
x = torch.zeros(1, 1, 1, 8)
for call in (lambda: dl.layer_norm_fwd(x), lambda: dl.attn_bwd(x, x, x, x, x, x), binding.load_calls):
    try:
        call()
    except ImportError as e:
        assert "/nowhere/dit_calls.so" in str(e)
    else:
        raise AssertionError("not refused")
print("fine")
"""
_LATE = """
from dit_long_sequence_gb300 import binding
loaded = lambda: "dit_calls-torch" in open("/proc/self/maps").read()
assert not loaded()
binding.load_calls()
assert loaded()
print("fine")
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    from dit_long_sequence_gb300 import build
    build.build()


@pytest.mark.parametrize("program", [_WITHOUT, _LATE], ids=["absent", "loaded late"])
def test_the_other_calls_do_without_it(program):
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_the_library_is_built_without_it(monkeypatch, tmp_path):
    from dit_long_sequence_gb300 import build

    def fails():
        raise RuntimeError("no such header")
    monkeypatch.setattr(build, "calls_path", lambda: str(tmp_path / "absent.so"))
    monkeypatch.setattr(build, "build_calls", fails)
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert build.build() == build.LIB


def test_its_file_is_of_one_pytorch_and_python(monkeypatch):
    import torch

    from dit_long_sequence_gb300 import build
    here = build.calls_path()
    assert torch.__version__ in here and sys.implementation.cache_tag in here and os.path.exists(here)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert build.calls_path() != here
