"""Tensors and streams of another device than the current one are refused by the packed cache's calls before anything is
launched (no GPU needed: the tensors only say where they lie)."""
import types

import pytest
import torch

import verify_sampling_gb300 as vs
from verify_sampling_gb300 import target

I32, F32, F64, U8 = torch.int32, torch.float32, torch.float64, torch.uint8


class Placed(torch.Tensor):
    """A host tensor that says it lies on CUDA device ``at``."""
    at = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.at


def _on(at, t):
    t = t.as_subclass(Placed)
    t.at = at
    return t


def _z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def _calls():
    """Each call with its tensors by name."""
    pairs = {"kd": _z(4, 1, 1, 4, 16, dtype=U8), "ks": _z(4, 1, 4, 1, dtype=U8), "vd": _z(4, 1, 1, 4, 16, dtype=U8),
             "vs": _z(4, 1, 4, 1, dtype=U8)}
    rows = {"q": _z(2, 2, 32), "q_out": _z(2, 2, 32), "k": _z(2, 1, 32), "v": _z(2, 1, 32), "freq": _z(16, dtype=F64),
            "position": _z(2, dtype=I32), "slot": _z(2, dtype=I32), "status": _z(1, dtype=I32), "q_weight": _z(32), "k_weight": _z(32)}

    def norm(d, kc, vc, **kw):
        return vs.norm_rope_cache(d["q"], d["k"], d["v"], d["freq"], d["position"], d["slot"], kc, vc, q_weight=d["q_weight"],
                                  k_weight=d["k_weight"], q_out=d["q_out"], status=d["status"], **kw)

    def read(d, **kw):
        return vs.cache_read_packed((d["kd"], d["ks"]), (d["vd"], d["vs"]), d["slot"], out=(d["k"], d["v"]), status=d["status"], **kw)

    def attend(d, **kw):
        return vs.prefix_attention_packed(d["q"], (d["kd"], d["ks"]), (d["vd"], d["vs"]), d["row_off"], d["kv_len"], d["block_table"],
                                          group_off=d["group_off"], prefix_len=d["prefix_len"], prefix_table=d["prefix_table"], out=d["q_out"],
                                          lse=d["lse"], workspace=d["workspace"], status=d["status"], want_lse=True, **kw)

    tables = {k: _z(*n, dtype=I32) for k, n in {"row_off": (3,), "kv_len": (2,), "block_table": (2, 3), "group_off": (2,), "prefix_len": (1,),
                                                 "prefix_table": (1, 2)}.items()}
    return {
        "norm": (lambda d, **kw: norm(d, d["k_cache"], d["v_cache"], **kw), {**rows, "k_cache": _z(4, 4, 1, 32), "v_cache": _z(4, 4, 1, 32)}),
        "append": (lambda d, **kw: norm(d, (d["kd"], d["ks"]), (d["vd"], d["vs"]), **kw), {**rows, **pairs}),
        "read": (read, {**pairs, **{k: rows[k] for k in ("k", "v", "slot", "status")}}),
        "attend": (attend, {**pairs, **tables, **{k: rows[k] for k in ("q", "q_out", "status")}, "lse": _z(2, 2),
                            "workspace": _z(1 << 20, dtype=U8)})}


class Reached(Exception):
    pass


@pytest.fixture
def no_launch(monkeypatch):
    """The current device is 0; a call that gets as far as the library raises Reached."""
    def stop(self, stream, *values):
        raise Reached

    monkeypatch.setattr(target._Call, "__call__", stop)
    monkeypatch.setattr(target, "_device", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(target, "_made", lambda stream: target._HERE)


@pytest.mark.parametrize("name", list(_calls()))
def test_every_tensor_has_to_lie_on_the_current_device(name, no_launch):
    call, tensors = _calls()[name]
    with pytest.raises(Reached):
        call({k: _on(0, t) for k, t in tensors.items()})
    for far in tensors:
        with pytest.raises(ValueError, match="current device"):
            call({k: _on(int(k == far), t) for k, t in tensors.items()})
    with pytest.raises(ValueError, match="current device"):
        call({k: _on(1, t) for k, t in tensors.items()})


@pytest.mark.parametrize("name", list(_calls()))
def test_a_stream_of_another_device_is_refused(name, no_launch):
    call, tensors = _calls()[name]
    tensors = {k: _on(0, t) for k, t in tensors.items()}
    for index, err in ((0, Reached), (1, ValueError)):
        with pytest.raises(err):
            call(tensors, stream=types.SimpleNamespace(cuda_stream=7, device=torch.device("cuda", index)))
