"""Tensors and streams of another device than the current one are refused before anything is launched (no GPU needed:
the tensors only say where they lie)."""
import types

import pytest
import torch

import verify_sampling_gb300 as vs
from verify_sampling_gb300 import target

I32, F32, F64 = torch.int32, torch.float32, torch.float64


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


def _z(*shape, dtype=I32):
    return torch.zeros(*shape, dtype=dtype)


def _calls():
    """Each call with its tensors by name."""
    cache = {"kv_len": _z(2), "block_table": _z(2, 3), "ring": _z(4)}
    made = {"new_len": _z(2), "position": _z(2), "request": _z(2), "slot": _z(2), "out_pos": _z(2, dtype=torch.int64)}

    def of(d):
        return {**{k: d[k] for k in cache}, "ring_pos": d["pos"], "page_size": 4}

    def reserve(d, **kw):
        out = {**{k: d[k] for k in made}, "ring_pos": d["out_pos"]}
        return vs.cache_reserve(of(d), d["row_off"], 2, pos_base=d["pos_base"], out=out, status=d["status"], **kw)

    def commit(d, **kw):
        res = {"new_len": d["new_len"], "ring_pos": d["pos"]}
        out = {"kv_len": d["out_len"], "ring_pos": d["out_pos"]}
        return vs.cache_commit(of(d), res, d["keep"], out=out, status=d["status"], **kw)

    def rope(d, **kw):
        return vs.rope_cache(d["q"], d["k"], d["v"], d["freq"], d["position"], d["slot"], d["k_cache"], d["v_cache"], q_out=d["q_out"],
                             status=d["status"], **kw)

    def attention(d, **kw):
        return vs.prefix_attention(d["q"], d["k_cache"], d["v_cache"], d["row_off"], d["kv_len"], d["block_table"], group_off=d["group_off"],
                                   prefix_len=d["prefix_len"], prefix_table=d["prefix_table"], out=d["q_out"], lse=d["lse"],
                                   workspace=d["workspace"], status=d["status"], want_lse=True, **kw)

    def logits(d, **kw):
        return vs.adjust_logits(d["logits"], d["tokens"], d["prompt_len"], d["length"], row_off=d["row_off"], x=d["x"], repetition=d["rep"],
                                frequency=d["freq"], presence=d["pres"], bias=(d["boff"], d["btok"], d["bval"]), mask=d["mask"],
                                mask_row=d["mask_row"], out=d["out"], status=d["status"], **kw)

    heads, page = dict(q=_z(2, 2, 8, dtype=F32), q_out=_z(2, 2, 8, dtype=F32)), _z(4, 4, 1, 8, dtype=F32)
    f = lambda *n: _z(*n, dtype=F32)  # noqa: E731
    return {
        "reserve": (reserve, {**cache, **made, "pos": _z(2, dtype=torch.int64), "row_off": _z(3), "pos_base": _z(2), "status": _z(1)}),
        "commit": (commit, {**cache, "new_len": _z(2), "pos": _z(2, dtype=torch.int64), "keep": _z(2), "out_len": _z(2),
                            "out_pos": _z(2, dtype=torch.int64), "status": _z(1)}),
        "rope": (rope, {**heads, "k": f(2, 1, 8), "v": f(2, 1, 8), "freq": _z(4, dtype=F64), "position": _z(2), "slot": _z(2),
                        "k_cache": page, "v_cache": page.clone(), "status": _z(1)}),
        "attention": (attention, {**heads, "k_cache": page, "v_cache": page.clone(), "row_off": _z(3), "kv_len": _z(2), "block_table": _z(2, 3),
                                  "group_off": _z(2), "prefix_len": _z(1), "prefix_table": _z(1, 2), "lse": f(2, 2),
                                  "workspace": _z(1 << 20, dtype=torch.uint8), "status": _z(1)}),
        "logits": (logits, {"logits": f(2, 9), "tokens": _z(2, 3), "prompt_len": _z(2), "length": _z(2), "row_off": _z(3), "x": _z(2, 2),
                            "rep": f(2), "freq": f(2), "pres": f(2), "boff": _z(3), "btok": _z(1), "bval": f(1), "mask": _z(2, 1),
                            "mask_row": _z(2), "out": f(2, 9), "status": _z(1)})}


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
