"""The package beside its library alone, as another torch or Python finds it: the prefill works,
the calls through the compiled binding say what is missing, and a binding that was built for
another torch is never loaded (CPU only)."""
import os
import subprocess
import sys

import pytest
import torch

import block_sparse_long_prefill_b200 as moba
from block_sparse_long_prefill_b200 import build

PKG = os.path.dirname(os.path.abspath(moba.__file__))


@pytest.mark.parametrize("stale", [None, "_binding.so", "_binding-1.0.0.so"])
def test_the_prefill_needs_the_library_alone(tmp_path, stale):
    pkg = tmp_path / os.path.basename(PKG)
    pkg.mkdir()
    for f in ("__init__.py", "build.py", "libmoba.so"):
        os.symlink(os.path.join(PKG, f), pkg / f)
    if stale:
        (pkg / stale).write_bytes(b"not a module")
    code = """
import torch, block_sparse_long_prefill_b200 as moba
assert moba.workspace_size(1, 4, 1, 1024, 64, 128, 3) > 0
x = torch.zeros(1, 2, 5, 64, dtype=torch.bfloat16)
t, i = x[0].transpose(0, 1), torch.zeros(5, 1, dtype=torch.int32)
for call, error, text in ((lambda: moba.swa_attn_fwd(x, x, x, 3), ValueError, "q must be a CUDA tensor"),
                          (lambda: moba.paged_decode_attn(t, x, x, i, i[:, 0]), ImportError, "build.py")):
    try:
        call()
    except error as e:
        assert text in str(e), e
    else:
        raise AssertionError(text)
"""
    subprocess.run([sys.executable, "-c", code], cwd=tmp_path, check=True, timeout=300)


def test_the_binding_is_named_for_its_torch(monkeypatch):
    path = build.binding_path()
    assert torch.__version__ in os.path.basename(path) and os.path.exists(path)
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    assert not os.path.exists(build.binding_path())
