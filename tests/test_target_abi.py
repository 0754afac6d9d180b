"""The argument structs of the target-model operators match the C layout, and bad
calls are refused on the host before any CUDA work (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest

import verify_sampling_gb300 as vs
from verify_sampling_gb300 import target

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"spec_cache_reserve_args": target.CacheReserveArgs,
           "spec_cache_commit_args": target.CacheCommitArgs,
           "spec_rope_cache_args": target.RopeCacheArgs,
           "spec_prefix_attention_args": target.PrefixAttentionArgs,
           "spec_logits_args": target.LogitsArgs}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(vs.LIB_PATH):
        from verify_sampling_gb300 import build
        build.build()
    return vs.lib()


def test_every_field_sits_where_c_puts_it(tmp_path):
    lines = []
    for c, cls in STRUCTS.items():
        lines.append(f'printf("{c} %zu\\n", sizeof({c}));')
        lines += [f'printf("{c}.{f[0]} %zu\\n", offsetof({c}, {f[0]}));' for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spec.h"\nint main(void){'
                   + "\n".join(lines) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    for c, cls in STRUCTS.items():
        assert int(got[c]) == ctypes.sizeof(cls), c
        for f in cls._fields_:
            assert int(got[f"{c}.{f[0]}"]) == getattr(cls, f[0]).offset, (c, f[0])


def test_packed_bytes_are_the_struct():
    for call in (target._RESERVE, target._COMMIT, target._ROPE, target._ATTENTION, target._LOGITS):
        values = [i + 1.5 if k is ctypes.c_float else i + 1 for i, (_, k) in enumerate(call.cls._fields_)]
        got = call.cls.from_buffer_copy(call.pack(*values))
        assert [getattr(got, f[0]) for f in call.cls._fields_] == values, call.name


def _filled(cls, **sizes):
    """Every pointer at an address of its own (never read: the calls under test are refused)."""
    a = cls()
    for i, (name, kind) in enumerate(cls._fields_):
        if kind is ctypes.c_void_p:
            setattr(a, name, 4096 * (i + 1))
    for name, v in sizes.items():
        setattr(a, name, v)
    return a


def _refusals(f, cls, sizes, cases):
    assert f(None, None) == vs.SPEC_ERR_INVALID_ARG
    for change, code in cases:
        a = _filled(cls, **{**sizes, **change})
        assert f(ctypes.byref(a), None) == code, change


BAD, ALIGN, UNSUP = vs.SPEC_ERR_INVALID_ARG, vs.SPEC_ERR_ALIGNMENT, vs.SPEC_ERR_UNSUPPORTED


def test_cache_calls_refuse(lib):
    sizes = dict(R=4, rows=16, page_size=16, n_pages=64, max_pages=8)
    common = [({"R": -1}, BAD), ({"R": 65536}, BAD), ({"page_size": 0}, BAD), ({"n_pages": 0}, BAD),
              ({"max_pages": 0}, BAD), ({"page_size": 1 << 20, "n_pages": 1 << 11}, BAD),
              ({"kv_len": None}, BAD), ({"block_table": None}, BAD), ({"ring": None}, BAD),
              ({"ring_pos": None}, BAD), ({"ring_out": None}, BAD), ({"ring_out": 4096, "ring_pos": 4096}, BAD),
              ({"ring_pos": 4100}, ALIGN), ({"block_table": 4098}, ALIGN), ({"status": 4097}, ALIGN)]
    _refusals(lib.spec_cache_reserve, target.CacheReserveArgs, sizes, common + [
        ({"rows": -1}, BAD), ({"row_off": None}, BAD), ({"new_len": None}, BAD), ({"slot": None}, BAD),
        ({"kv_len": 8192, "new_len": 8192}, BAD), ({"position": 4099}, ALIGN)])
    sizes.pop("rows")
    _refusals(lib.spec_cache_commit, target.CacheCommitArgs, sizes, common + [
        ({"keep": None}, BAD), ({"kv_out": None}, BAD), ({"kv_out": 8192, "keep": 8192}, BAD),
        ({"kv_out": 4098}, ALIGN)])


def test_rope_refuses(lib):
    sizes = dict(rows=4, Hq=8, Hk=2, D=64, rot=64, n_slots=100)
    _refusals(lib.spec_rope_cache, target.RopeCacheArgs, sizes, [
        ({"rows": -1}, BAD), ({"Hq": -1}, BAD), ({"Hk": 1025}, BAD), ({"D": 0}, BAD), ({"rot": 63}, BAD),
        ({"rot": 66}, BAD), ({"rot": -2}, BAD), ({"dtype": 2}, BAD), ({"layout": 2}, BAD), ({"D": 514}, UNSUP),
        ({"q": None}, BAD), ({"q_out": None}, BAD), ({"k": None}, BAD), ({"v_cache": None}, BAD), ({"slot": None}, BAD),
        ({"freq": None}, BAD), ({"position": None}, BAD), ({"n_slots": 0}, BAD), ({"q": 4098}, ALIGN),
        ({"freq": 4100}, ALIGN), ({"slot": 4098}, ALIGN), ({"dtype": 1, "k_cache": 4097}, ALIGN)])
    # nothing to do: nothing is launched
    assert lib.spec_rope_cache(ctypes.byref(_filled(target.RopeCacheArgs, **{**sizes, "rows": 0})), None) == vs.SPEC_OK


def test_rope_frequencies():
    import math

    import torch
    f, scale = vs.rope_frequencies(64, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and scale == 1.0
    assert torch.allclose(f, torch.tensor([10000.0 ** (-i / 32) for i in range(32)], dtype=torch.float64), rtol=1e-14)
    lin, _ = vs.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(lin, f / 4)
    b, _ = vs.rope_frequencies(64, scaling="base", factor=8.0, device="cpu")
    assert b[0] == f[0] and abs(b[-1] / (f[-1] / 8) - 1) < 1e-12
    for kind in ("ramp", "band"):
        s, scale = vs.rope_frequencies(64, scaling=kind, factor=8.0, trained=4096, low=1.0, high=32.0, device="cpu")
        turns = 4096 * f / (2 * math.pi)
        assert torch.equal(s[turns > 64], f[turns > 64]) and torch.allclose(s[turns < 0.5], f[turns < 0.5] / 8, rtol=1e-14)
        assert torch.all((s <= f) & (s >= f / 8)) and torch.all(s.diff() <= 0)
        assert scale == (1.0 if kind == "band" else 0.1 * math.log(8.0) + 1.0)
    for bad in (dict(rot=7), dict(rot=64, factor=0.5), dict(rot=64, scaling="ramp"), dict(rot=64, scaling="other")):
        with pytest.raises(ValueError):
            vs.rope_frequencies(device="cpu", **bad)


def test_logits_refuse(lib):
    sizes = dict(R=4, V=100, rows=8, rows_per_request=2, ld=100, out_ld=128, tokens_ld=50, tokens_cols=50, x_ld=3, x_cols=3,
                 n_bias=10, mask_ld=4, n_masks=2)
    _refusals(lib.spec_adjust_logits, target.LogitsArgs, sizes, [
        ({"R": -1}, BAD), ({"R": 65536}, BAD), ({"V": 0}, BAD), ({"V": 1 << 30}, BAD), ({"rows": -1}, BAD), ({"dtype": 2}, BAD),
        ({"logits": None}, BAD), ({"out": None}, BAD), ({"ld": 99}, BAD), ({"out_ld": 99}, BAD),
        ({"logits": 4096, "out": 4096}, BAD), ({"row_off": None, "rows_per_request": 3}, BAD),
        ({"row_off": None, "rows_per_request": -1}, BAD), ({"tokens": None}, BAD), ({"length": None}, BAD),
        ({"tokens_cols": 51}, BAD), ({"tokens_cols": -1}, BAD), ({"x_cols": 65, "x_ld": 65}, BAD), ({"x_cols": 4}, BAD),
        ({"bias_off": None}, BAD), ({"bias_val": None}, BAD), ({"n_bias": -1}, BAD), ({"mask_ld": 3}, BAD), ({"n_masks": 0}, BAD),
        ({"logits": 4098}, ALIGN), ({"dtype": 1, "out": 4097}, ALIGN), ({"tokens": 4097}, ALIGN), ({"mask": 4098}, ALIGN)])
    for none in ({"R": 0}, {"rows": 0}):
        assert lib.spec_adjust_logits(ctypes.byref(_filled(target.LogitsArgs, **{**sizes, **none})), None) == vs.SPEC_OK


def test_attention_refuses(lib):
    need = vs.attention_workspace_bytes(8, 4, 8, 64)
    assert need > 0 and vs.attention_workspace_bytes(-1, 4, 8, 64) == 0 and vs.attention_workspace_bytes(8, 4, 8, 257) == 0
    sizes = dict(R=4, rows=8, Hq=8, Hk=2, D=64, page_size=16, n_pages=20, max_pages=4, G=2, max_prefix_pages=3, scale=0.125,
                 workspace_bytes=need)
    _refusals(lib.spec_prefix_attention, target.PrefixAttentionArgs, sizes, [
        ({"R": -1}, BAD), ({"R": 65536}, BAD), ({"rows": -1}, BAD), ({"Hq": 0}, BAD), ({"Hq": 7}, BAD), ({"Hk": 0}, BAD),
        ({"Hq": 1026}, BAD), ({"D": 0}, BAD), ({"D": 257}, UNSUP), ({"dtype": 3}, BAD), ({"page_size": 0}, BAD), ({"n_pages": 0}, BAD),
        ({"max_pages": 0}, BAD), ({"G": -1}, BAD), ({"G": 5}, BAD), ({"max_prefix_pages": 0}, BAD), ({"scale": 0.0}, BAD),
        ({"scale": float("nan")}, BAD), ({"scale": float("inf")}, BAD), ({"q": None}, BAD), ({"k_cache": None}, BAD), ({"out": None}, BAD),
        ({"row_off": None}, BAD), ({"kv_len": None}, BAD), ({"block_table": None}, BAD), ({"group_off": None}, BAD),
        ({"prefix_table": None}, BAD), ({"rows": 1 << 30, "Hq": 2}, BAD), ({"q": 4098}, ALIGN), ({"lse": 4097}, ALIGN),
        ({"prefix_len": 4098}, ALIGN), ({"workspace": None}, vs.SPEC_ERR_WORKSPACE), ({"workspace_bytes": need - 1}, vs.SPEC_ERR_WORKSPACE),
        ({"workspace": 4096 + 128}, ALIGN)])
    for none in ({"R": 0, "G": 0}, {"rows": 0}):
        assert lib.spec_prefix_attention(ctypes.byref(_filled(target.PrefixAttentionArgs, **{**sizes, **none})), None) == vs.SPEC_OK
