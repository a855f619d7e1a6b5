"""_marshal.so on the CPU: who needs it, when it is built anew, and what its
functions make of arguments that only Python can get wrong."""
import os
import shutil
import subprocess
import sys
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_415_b200 import build
    build.build()
    from paged_kv_cache_415_b200 import binding
    return binding


def test_other_calls_do_not_need_it(pa, tmp_path):
    """A package with libpa.so alone imports and serves the calls that need
    no more; the others say what is missing."""
    dst = tmp_path / "paged_kv_cache_415_b200"
    shutil.copytree(os.path.join(ROOT, "paged_kv_cache_415_b200"), dst,
                    ignore=shutil.ignore_patterns("*.so", "__pycache__"))
    os.symlink(pa.LIB_PATH, dst / "libpa.so")
    code = ("from paged_kv_cache_415_b200 import binding as B, step\n"
            "assert B.pa_paged_decode_workspace_size(4, 8, 2, 128, 16, 100, 64) > 0\n"
            "assert B.pa_latent_decode_workspace_size(4, 16, 512, 16, 4096) > 0\n"
            "B.pa_rope_append(*[None] * 9)\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode != 0
    assert "ImportError: _marshal.so is not built" in res.stderr, res.stderr[-500:]
    assert "binding.py" in res.stderr and "pa_rope_append" in res.stderr


def test_one_built_for_another_torch_is_refused(pa, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.raises(ImportError, match="9.9.9"):
        pa._Marshal().rope_append
    monkeypatch.undo()
    assert pa._Marshal().rope_append


def test_built_anew_for_another_python_or_torch(pa, monkeypatch, tmp_path):
    from paged_kv_cache_415_b200 import build
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "MARSHAL_KEY", str(tmp_path / "key"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)
    build.build_marshal()
    build.build_marshal()
    assert len(runs) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build_marshal()
    build.build_marshal()
    assert len(runs) == 2 and '-DPA_TORCH_VERSION="9.9.9"' in runs[1]
    os.remove(tmp_path / "key")                      # built before there was a record
    build.build_marshal()
    assert len(runs) == 3


def test_a_flag_that_is_neither_true_nor_false_is_refused(pa):
    t, h = torch.zeros, torch.float16
    long = t(4, dtype=torch.int64)
    rope = [t(4, 8, 128, dtype=h), t(4, 8, 128, dtype=h), t(4, 2, 128, dtype=h),
            t(4, 2, 128, dtype=h), t(3, 16, 2, 128, dtype=h), t(3, 16, 2, 128, dtype=h), long, long,
            t(10, 128)]
    latent = [None, None, t(4, 576, dtype=h), t(3, 16, 576, dtype=h), long, long, t(10, 64)]
    both = t(2).numpy()
    for call, args in ((pa.pa_rope_append, rope), (pa.pa_latent_append, latent)):
        with pytest.raises(ValueError, match="interleaved"):
            call(*args, interleaved=both)
        for flag in (0, 1, True, None):              # refused for the device alone
            with pytest.raises(ValueError, match="CUDA"):
                call(*args, interleaved=flag)
