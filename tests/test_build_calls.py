"""The compiled argument marshalling is optional: the library is built, and its calls are made, without it."""
import os
import subprocess
import sys
import types
import warnings

import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import blocks, build


@pytest.fixture
def dry(tmp_path, monkeypatch):
    """The build with compilers that write empty files, into a folder of its own."""
    for name in ("BUILD_DIR", "LIB_PATH", "CALLS_PATH", "ABLATION_PATH", "MFMA_FORM_PATH", "STREAM_CEILING_PATH", "KERNEL_TIMELINE_PATH"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    made = []

    def run(cmd, **kwargs):
        open(cmd[cmd.index("-o") + 1], "w").close()
        made.append(cmd)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    return made


def test_library_without_a_host_compiler(dry, monkeypatch):
    which = build.shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda name: None if name in ("g++", "c++") else which(name))
    open(build.CALLS_PATH, "w").close()                 # of an earlier build
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.KERNEL_TIMELINE_PATH) and not os.path.exists(build.CALLS_PATH)


def test_library_without_torch(dry, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(RuntimeWarning, match="marshalled in Python"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.CALLS_PATH)


def test_both_are_built(dry):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        build.build()
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.CALLS_PATH)


@pytest.mark.parametrize("how", ["missing", "of another torch"])
def test_calls_go_through_python_without_it(monkeypatch, how):
    other = None if how == "missing" else types.SimpleNamespace(torch_version="0.0")
    monkeypatch.setitem(sys.modules, "tiled_dense_gemm_relu_amd._blocks_calls", other)
    if other is None:
        monkeypatch.delattr(gr, "_blocks_calls", raising=False)
    else:
        monkeypatch.setattr(gr, "_blocks_calls", other, raising=False)
    monkeypatch.setattr(blocks, "_calls", None)
    with pytest.warns(RuntimeWarning, match="build the package again"):
        with pytest.raises(ValueError, match="GPU tensor"):      # Python's own refusal: the call got that far
            gr.quantize_blocks(torch.zeros((2, 2), dtype=torch.float16))
    with warnings.catch_warnings():
        warnings.simplefilter("error")                            # said once
        with pytest.raises(ValueError, match="GPU tensor"):
            gr.quantize_blocks(torch.zeros((2, 2), dtype=torch.float16))


def test_the_built_one_is_of_this_torch():
    code = "import torch, tiled_dense_gemm_relu_amd.blocks as b; c = b._compiled(); assert c.torch_version == torch.__version__"
    subprocess.run([sys.executable, "-W", "error::RuntimeWarning", "-c", code], check=True, cwd=build.ROOT)
