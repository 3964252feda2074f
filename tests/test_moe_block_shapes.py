"""The example block refuses tensors that its buffers and the library's row counts do not fit, before any call
of the library (no GPU)."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
block = importlib.util.module_from_spec(spec)
spec.loader.exec_module(block)

H, T = 128, 4


class Called(Exception):
    pass


class Library:
    """Stands for the library: a step that reaches it has accepted its tensors."""

    def __getattr__(self, name):
        def f(*args, **kw):
            raise Called(name)
        return f


def _rows(n=T, h=H, dtype=torch.bfloat16):
    return torch.zeros(n, h, dtype=dtype)


def _steps():
    """(name, step, its number of tensors) of the block's classes with buffers for T tokens."""
    out = []
    for name, cls, calls in (("serving", block.Serving, ["step"]), ("e4m3", block.ServingFp8, ["step"]),
                             ("training", block.Training, ["forward", "backward"])):
        b = cls.__new__(cls)   # without its device buffers
        b.H, b.T, b.cfg, b.norm, b.n = H, T, None, None, _rows()
        b.w = {"norm": None, "gate_w": None, "bias": None}
        for k in ("xq", "xs", "sum", "y", "tw", "pos"):
            setattr(b, k, _rows())
        out += [(name, getattr(b, c), 3 if c == "step" else 2) for c in calls]
    return out


@pytest.mark.parametrize("i", range(4))
def test_tensors_that_do_not_fit_are_refused(monkeypatch, i):
    monkeypatch.setattr(block, "moe", Library())
    name, step, n = _steps()[i]
    with pytest.raises(Called):
        step(*[_rows() for _ in range(n)])
    with pytest.raises(ValueError):
        step(*[_rows(T + 1) for _ in range(n)])            # more tokens than the buffers hold
    if name == "training":
        with pytest.raises(ValueError):
            step(*[_rows(T - 1) for _ in range(n)])        # a fixed number of tokens
    else:
        with pytest.raises(Called):
            step(*[_rows(T - 1) for _ in range(n)])
    wide = torch.zeros(T, 2 * H, dtype=torch.bfloat16)[:, :H]
    for j in range(n):
        for bad in (_rows(T + 1), _rows(T - 1), _rows(h=64), _rows(dtype=torch.float32), wide):
            with pytest.raises(ValueError):
                step(*[bad if j == k else _rows() for k in range(n)])
