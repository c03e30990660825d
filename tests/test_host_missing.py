"""The library and the package without the module _host: no torch or host compiler where the library is built, no _host,
or one for another torch, where the package is imported.  Serving calls are marshalled in Python then."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

from tests.conftest import ROOT

PACKAGE = "bit_group_quantized_q4gsw_amd"
CALLS = """
import warnings
with warnings.catch_warnings(record=True) as told:
    warnings.simplefilter("always")
    import bit_group_quantized_q4gsw_amd as q
import torch
assert [w for w in told if "marshalled in Python" in str(w.message)], told
assert q.packed_bytes(64, 64, 32, torch.float16) > 0
i, x = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 64)
c = q.KvCache(q.binding.KvCacheDesc(4, 32, 2, 64, 0, None, 0), torch.empty(0, dtype=torch.uint8))
s = q.Adapters(q.binding.AdaptersDesc(8, 8, 1, 4, q.BF16, 0, None, 0), torch.empty(0, dtype=torch.uint8))
where = (i[:2].view(1, 2), i[:2], i[:1])
for call in (lambda: q.logits_adjust(torch.zeros(3, 40)), lambda: q.kv_append(c, x, x.half(), *where),
             lambda: q.kv_attention(c, x[0], *where, 3, 3), lambda: q.kv_tree_attention(c, x, i[:2], *where, 3, 3),
             lambda: q.kv_keep(c, i.long(), i[:1], *where, 3), lambda: q.adapters_add(x[:, 0], torch.zeros(3, 9), s, i)):
    try:
        call()
    except ValueError:
        continue
    raise AssertionError("not refused")
print("ok")
"""


def package(folder, host=None):
    """The package in `folder`, its _host replaced by the text `host`, or gone."""
    to = folder / PACKAGE
    to.mkdir()
    for name in ("__init__.py", "binding.py"):
        shutil.copy(os.path.join(ROOT, PACKAGE, name), to / name)
    os.symlink(os.path.join(ROOT, PACKAGE, "libq4gsw.so"), to / "libq4gsw.so")
    if host is not None:
        (to / "_host.py").write_text(host)
    return folder


@pytest.mark.parametrize("host", [
    None, "raise ImportError('undefined symbol')", "torch_version = '0.1'\ndef open(*a): raise AssertionError('of another torch')",
    "import torch\ntorch_version = torch.__version__.split('+')[0]\ndef open(*a): raise ImportError('no such call')",
    "import torch\ntorch_version = torch.__version__.split('+')[0]\ndel torch._C._cuda_getDevice"])       # a torch without GPUs
def test_import_without_host(tmp_path, host):
    res = subprocess.run([sys.executable, "-c", CALLS], cwd=package(tmp_path, host), capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.strip().endswith("ok"), res.stdout + res.stderr


def builder(folder, monkeypatch):
    """build.py on a library of one small source in `folder`."""
    spec = importlib.util.spec_from_file_location("_small_build", os.path.join(ROOT, PACKAGE, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    (folder / "csrc").mkdir()
    (folder / "csrc" / "one.hip").write_text('extern "C" int one() { return 1; }\n')
    for name, to in dict(CSRC="csrc", LIB="lib.so", HOST="_host.so", BUILD_DIR="objects").items():
        monkeypatch.setattr(b, name, str(folder / to))
    return b


def test_build_without_torch(tmp_path, monkeypatch, capfd):
    b = builder(tmp_path, monkeypatch)
    (tmp_path / "_host.so").write_bytes(b"of another environment")
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    assert os.path.exists(b.build()) and not os.path.exists(b.HOST)
    assert "no torch" in capfd.readouterr().err


def test_build_without_a_host_compiler(tmp_path, monkeypatch, capfd):
    b = builder(tmp_path, monkeypatch)
    monkeypatch.setattr(b.shutil, "which", lambda name: None)
    assert os.path.exists(b.build()) and not os.path.exists(b.HOST)
    assert "no host compiler" in capfd.readouterr().err


def test_a_host_that_does_not_compile_is_told(tmp_path, monkeypatch):
    b = builder(tmp_path, monkeypatch)
    (tmp_path / "csrc" / "host.cpp").write_text("#error not today\n")
    with pytest.raises(RuntimeError, match="host.cpp"):
        b.build()
    assert os.path.exists(b.LIB)


def test_a_torch_between_releases(tmp_path):
    """Whose __version__ says more than the version that its headers give."""
    host = "import torch\ntorch_version = torch.__version__.split('+')[0]\ntorch.__version__ = torch_version + 'a0+git1'\ndef open(*a): pass\n"
    call = "import warnings\nwarnings.simplefilter('error', RuntimeWarning)\nimport bit_group_quantized_q4gsw_amd as q\nprint(q.binding._host.__name__)"
    res = subprocess.run([sys.executable, "-c", call], cwd=package(tmp_path, host), capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.strip().endswith("_host"), res.stdout + res.stderr
