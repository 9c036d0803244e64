"""CPU: the binding without its native front: it falls back on the checks in
Python, with one warning, and the build leaves no stale front beside a new
library."""

import sys
import warnings

import pytest
import torch

import mlp_fp8_quant_amd as fp8
from mlp_fp8_quant_amd import api, build as b


def without_front(monkeypatch):
    monkeypatch.setattr(api, "_native", None)
    monkeypatch.delattr(fp8, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "mlp_fp8_quant_amd._binding", None)   # importing it fails


def test_calls_fall_back_on_the_checks_in_python(monkeypatch):
    without_front(monkeypatch)
    q, s = torch.zeros(4, 16, dtype=torch.uint8), torch.ones(1)
    bf = torch.zeros(4, 16, dtype=torch.bfloat16)
    with warnings.catch_warnings(record=True) as seen:
        warnings.simplefilter("always")
        for call in (lambda: fp8.fp8_linear_act(q, q, s, s), lambda: fp8.fp8_layer_norm(bf),
                     lambda: fp8.fp8_linear_act_backward(bf, None),
                     lambda: fp8.fp8_layer_norm_backward(bf, bf, None, s, s)):
            with pytest.raises(ValueError, match="must be on a GPU"):
                call()
    assert [str(w.message) for w in seen].count(api.NO_FRONT) == 1


def test_the_front_is_used_where_it_is_built(monkeypatch):
    monkeypatch.setattr(api, "_native", None)
    front = api._load_native()
    assert front is api._native and front.__name__.endswith("_binding")


def test_build_without_a_host_compiler_removes_the_old_front(monkeypatch, tmp_path):
    old = tmp_path / "_binding.so"
    old.write_bytes(b"of another library")

    def fails(verbose=False):
        raise RuntimeError("command failed: g++")

    monkeypatch.setattr(b, "BINDING_PATH", str(old))
    monkeypatch.setattr(b, "build_binding", fails)
    with pytest.warns(UserWarning, match="native front"):
        b.build_front()
    assert not old.exists()
    with pytest.warns(UserWarning):
        b.build_front()                      # nothing there to remove
