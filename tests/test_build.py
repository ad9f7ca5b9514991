"""What the build makes of what is installed: the library needs no torch, and the package works without its extension module."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LOAD = f"""
import importlib.util, os, sys
spec = importlib.util.spec_from_file_location("build", {os.path.join(ROOT, "mxfp4_weight_mxfp8_gb300", "build.py")!r})
build = importlib.util.module_from_spec(spec)
spec.loader.exec_module(build)
"""


def python(code, *flags, **env):
    run = subprocess.run([sys.executable, *flags, "-c", code], cwd=ROOT, env=dict(os.environ, **env), capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
    return run.stdout


@pytest.fixture()
def compiler(tmp_path):
    """A stand-in for nvcc that makes empty outputs: {variables} for a build in a folder of its own."""
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.parent.mkdir()
    nvcc.write_text('#!/bin/sh\nwhile [ "$1" != "-o" ]; do shift; done\n: > "$2"\n')
    nvcc.chmod(0o755)
    (nvcc.parent / "g++").symlink_to(nvcc)
    return dict(NVCC=str(nvcc), MOE_BUILD_DIR=str(tmp_path / "made"))


@pytest.fixture()
def bare_library(tmp_path):
    """The library in a folder without the extension module."""
    import __graft_entry__

    __graft_entry__.build()
    import mxfp4_weight_mxfp8_gb300 as moe

    library = tmp_path / "libmoe_gb300.so"
    library.symlink_to(moe.library()._name)
    return str(library)


def test_the_library_is_built_where_torch_is_not_installed(compiler, tmp_path):
    code = LOAD + """
assert importlib.util.find_spec("torch") is None and not build.up_to_date()
assert os.path.exists(build.build()) and build.up_to_date()
"""
    python(code, "-I", "-S", **compiler)
    assert "libmoe_gb300.so" in os.listdir(tmp_path / "made") and not [f for f in os.listdir(tmp_path / "made") if f.startswith("_tensors")]


def test_an_extension_module_of_another_torch_is_not_up_to_date(compiler, tmp_path):
    (tmp_path / "torch" / "lib").mkdir(parents=True)
    for f in ("__init__.py", "lib/libc10_cuda.so"):
        (tmp_path / "torch" / f).touch()
    code = f"import sys\nsys.path.insert(0, {str(tmp_path)!r})\n" + LOAD + """
assert build.up_to_date() == (sys.argv[1:] == ["built"])
build.build()
assert build.up_to_date() and os.path.exists(build.TENSORS)
print(build.TENSORS)
"""
    def made(version, *args):
        (tmp_path / "torch" / "version.py").write_text(f"__version__ = '{version}'\n")
        return python(code.replace("sys.argv[1:]", repr(list(args))), "-I", "-S", PATH=f"{tmp_path / 'bin'}:{os.environ['PATH']}", **compiler)

    first, second = made("9.1.0+cu999"), made("9.2.0")
    assert first != second and made("9.1.0+cu999", "built") == first


def test_calls_without_the_extension_module_are_checked_by_the_package(bare_library):
    code = """
import torch
import mxfp4_weight_mxfp8_gb300 as moe
x, ids = torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32)
for call in (lambda: moe.moe_route(x, ids, torch.zeros(2, 2)), lambda: moe.moe_norm(x, x[0], x), lambda: moe.moe_rope(ids[0], ids, x.bfloat16()),
             lambda: moe.moe_kv_copy((x, x, x, x), ids)):
    try:
        call()
    except moe.MoeError as e:
        assert e.code == moe.MOE_ERR_ARG and "current CUDA device" in str(e), e
    else:
        raise SystemExit("taken")
print(moe.library()._name)
"""
    assert python(code, MOE_LIBRARY=bare_library).strip() == bare_library


@pytest.mark.gpu
def test_calls_without_the_extension_module_give_the_same_bits(bare_library, tmp_path):
    code = """
import sys
import torch
import mxfp4_weight_mxfp8_gb300 as moe
g = torch.Generator(device="cuda").manual_seed(3)
x, w = torch.randn(5, 256, generator=g, device="cuda").to(torch.bfloat16), torch.randn(256, generator=g, device="cuda")
out, codes, scales = torch.empty_like(x), torch.empty(5, 256, dtype=torch.uint8, device="cuda"), torch.empty(5, 8, dtype=torch.uint8, device="cuda")
moe.moe_norm(x, w, out, codes=codes, scales=scales)
q = torch.randn(5, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
moe.moe_rope(torch.arange(5, dtype=torch.int32, device="cuda"), moe.moe_rope_turns(64, device="cuda"), q)
ids, weights = torch.empty(5, 16, dtype=torch.int32, device="cuda"), torch.empty(5, 16, device="cuda")
moe.moe_route(x.float(), ids, weights)
moe.moe_norm(x, w, out, codes=codes, scales=scales)
torch.save([t.cpu() for t in (out, codes, scales, q, ids, weights)], sys.argv[1])
print(type(moe._native).__name__)
"""
    import torch

    results = []
    for name, env in (("bare", dict(MOE_LIBRARY=bare_library)), ("whole", {})):
        path = str(tmp_path / name)
        kind = python("import sys\nsys.argv = ['', %r]\n" % path + code, **env).strip()
        assert (kind == "module") == (name == "whole")
        results.append(torch.load(path))
    assert all(torch.equal(a, b) for a, b in zip(*results))
