"""The compiled binding's refusals of tensors (no GPU, no launch)."""
import os
import types

import pytest
import torch

import routed_expert_ffn_04_gb300 as moe


@pytest.fixture(scope="module", autouse=True)
def lib():
    return moe.load(build_if_missing=True)


H = types.SimpleNamespace(address=None, device=0)
X = torch.zeros(4, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("x, text", [(X, "on cuda:0, got .* cpu"), (X.float(), "dense torch.bfloat16"), (None, "x is missing"),
                                     (X[:, :0], "at least one column"), (X[0, 0], "at least one column")])
def test_refused_x(x, text):
    with pytest.raises(moe.MoEError, match=text) as e:
        moe.add_rmsnorm(H, x, X[0], 1e-5, out=X)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG


def test_every_function_refuses_host_tensors():
    c = moe.make_config(4, 64, 8, 2, 64, 64, 1.0)
    f = torch.zeros(4, 8)
    for call in (lambda: moe.add_rmsnorm_backward(H, X, X, X[0], f[:, 0], X),
                 lambda: moe.combine_backward(H, c, X, f, f, f, X, f), lambda: moe.route_backward(H, c, f, f, f, f),
                 lambda: moe.permute_backward(H, c, X, f, X),
                 lambda: moe.grouped_swiglu_backward(H, X, X, None, X, X, X, X, X, X, X, None, num_groups=1, H=64, I=64)):
        with pytest.raises(moe.MoEError) as e:
            call()
        assert e.value.status == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(num_groups=-1, H=64, I=64), dict(num_groups=1, H=32, I=64),
                                dict(num_groups=2**31 - 1, H=64, I=64), dict(num_groups=1, H=64, I=2**40)])
def test_grouped_sizes(kw):
    with pytest.raises(moe.MoEError) as e:
        moe.grouped_swiglu_backward(H, X, X, None, X, X, X, X, X, X, X, None, **kw)
    assert e.value.status == moe.MOE_ERR_INVALID_ARG


def test_arguments_of_other_kinds():
    with pytest.raises(TypeError):
        moe.add_rmsnorm(H, X, X[0], "eps")
    with pytest.raises(TypeError):
        moe.permute_backward(H, None, X, X, X)  # not a Config
    with pytest.raises(AttributeError):
        moe.add_rmsnorm(H, [1.0], X[0], 1e-5)


def test_the_layer_loads_without_the_binding(monkeypatch, tmp_path):
    monkeypatch.setattr(moe, "_lib", None)
    monkeypatch.setattr(moe, "_native_module", None)
    monkeypatch.setattr(moe._build, "BINDING", str(tmp_path / "_binding.so"))
    assert moe.load() is not None and moe.status_string(0) == "ok"
    assert moe.workspace_size(moe.make_config(4, 64, 8, 2, 64, 64, 1.0)) > 0
    with pytest.raises(ImportError, match="_binding.so is missing"):
        moe.add_rmsnorm(H, X, X[0], 1e-5, out=X)


def test_the_library_builds_without_python_headers(monkeypatch, tmp_path):
    moe._build.build()  # the library is of these sources
    target = tmp_path / "_binding.so"
    target.write_bytes(b"of an older source")
    os.utime(target, (0, 0))
    monkeypatch.setattr(moe._build, "BINDING", str(target))
    monkeypatch.setattr(moe._build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    before = os.path.getmtime(moe._build.LIB)
    with pytest.warns(UserWarning, match="Python.h"):
        assert moe._build.build() == moe._build.LIB
    assert not target.exists() and os.path.getmtime(moe._build.LIB) == before


def test_the_binding_builds_alone(monkeypatch, tmp_path):
    """For another interpreter beside a library that is there."""
    moe._build.build()
    target = tmp_path / "_binding.so"
    monkeypatch.setattr(moe._build, "BINDING", str(target))
    before = os.path.getmtime(moe._build.LIB)
    moe._build.build()
    assert target.exists() and os.path.getmtime(moe._build.LIB) == before
