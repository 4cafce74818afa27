"""The library builds, and the decode-step calls are made, without a C compiler or
Python's headers (CPU; stand-ins for CUDA tensors and a launch failure armed)."""
import importlib
import os

import pytest

torch = pytest.importorskip("torch")

import hadamard_rotated_activation_b200 as kq
from hadamard_rotated_activation_b200 import build as kqbuild
from test_decode_cache import Array, _attn, _cache, _copy
from test_decode_call import BF, F16, F32, U8


@pytest.mark.parametrize("lacks", ["compiler", "headers"])
def test_build_without(lacks, monkeypatch, tmp_path, capsys):
    kqbuild.build()
    call = tmp_path / "_kq_call.so"
    monkeypatch.setattr(kqbuild, "CALL", str(call))
    if lacks == "compiler":
        monkeypatch.setattr(kqbuild.shutil, "which", lambda name: None)
    else:
        monkeypatch.setattr(kqbuild.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert kqbuild.build_call() is None and kqbuild.build() == kqbuild.LIB
    assert lacks in capsys.readouterr().err
    # one of an older source does not stay
    call.write_bytes(b"")
    os.utime(call, (1, 1))
    assert kqbuild.build() == kqbuild.LIB and not call.exists()


def test_build_call_builds(monkeypatch, tmp_path):
    call = tmp_path / "_kq_call.so"
    monkeypatch.setattr(kqbuild, "CALL", str(call))
    assert kqbuild.build_call() == str(call) and call.stat().st_size > 0


def test_calls_without_the_module(monkeypatch):
    kqbuild.build()
    L = kq.lib()

    def missing(name, package=None):
        raise ImportError(name)
    monkeypatch.setattr(kq, "_call", None)
    monkeypatch.setattr(importlib, "import_module", missing)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    def gemv(stream=0, **change):
        a = dict(x=Array(BF, 2, 256), codes=Array(U8, 100, 128), scales=Array(F16, 100, 2),
                 zeros=Array(F16, 100, 2), tensor_scale=None, group=128, y=Array(F32, 2, 100))
        kq.kq_gemv(kq.KQ_FMT_INT4_ASYM, **{**a, **change}, stream=stream)
    try:
        with pytest.warns(RuntimeWarning):
            L.kq_diag_fail_next_launch(701)
            with pytest.raises(kq.KQError) as e:
                gemv()
        assert e.value.status == kq.KQ_ERR_CUDA
        for call in (lambda: _attn(_cache(), _cache()), lambda: _copy(_cache(2), _cache(2))):
            L.kq_diag_fail_next_launch(701)
            with pytest.raises(kq.KQError) as e:
                call()
            assert e.value.status == kq.KQ_ERR_CUDA
        with pytest.raises(ValueError):
            gemv(y=Array(F32, 2, 99))
    finally:
        L.kq_diag_fail_next_launch(0)
