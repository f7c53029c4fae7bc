"""The quantized layers need libsvdq.so alone: without the extension behind the
16-bit operators the package imports and packs, and those operators say what
is missing; and a failed build of it leaves libsvdq.so installed."""

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

import bit_quantized_diffusion_amd as bq

PKG = os.path.dirname(os.path.abspath(bq.__file__))

SCRIPT = """
import numpy as np, torch
import bit_quantized_diffusion_amd as bq
packed = bq.pack_weights(np.full((32, 64), 0x3F80, np.uint16), np.full(64, 4.0, np.float32), 16)
assert packed["wq"].size
assert bq.attention_workspace_size(1, 8192, 1, 8, 8, 128) > 0
x = torch.zeros(4, 64, dtype=torch.bfloat16)
for call in (lambda: bq.layer_norm(x), lambda: bq.linear16(x, x), lambda: bq.attention(x[None], x[None], x[None])):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e)
    else:
        raise AssertionError("ran without its extension")
print("quantized layers alone")
"""


def test_package_without_the_extension(tmp_path):
    copy = tmp_path / "bit_quantized_diffusion_amd"
    copy.mkdir()
    for f in os.listdir(PKG):
        if f.endswith(".py") or f == "libsvdq.so":
            shutil.copy(os.path.join(PKG, f), copy / f)
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=tmp_path, capture_output=True, text=True,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0 and "quantized layers alone" in r.stdout, r.stdout + r.stderr


def _build_module(tmp_path):
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.LIB = str(tmp_path / "libsvdq.so")
    mod.PYTHON_LIB = str(tmp_path / os.path.basename(mod.PYTHON_LIB))
    mod.KERNEL_SOURCES = []      # the host sources compile in a second; nothing is loaded
    return mod


def test_extension_is_named_for_its_python():
    spec = importlib.util.spec_from_file_location("_build_named", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert os.path.basename(mod.PYTHON_LIB) == "_block_ops" + sysconfig.get_config_var("EXT_SUFFIX")


def test_a_failed_extension_leaves_the_library_installed(tmp_path, capsys):
    mod = _build_module(tmp_path)
    mod.PYTHON_SOURCE = "not_there.cpp"
    with pytest.raises(RuntimeError):
        mod.build()
    assert os.path.exists(mod.LIB) and not os.path.exists(mod.PYTHON_LIB)
