"""The argument structs of the packed cache's calls match the C layout, and bad calls are refused on the host (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest

import verify_sampling_gb300 as vs
from verify_sampling_gb300 import target

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD, ALIGN, UNSUP, WORK = vs.SPEC_ERR_INVALID_ARG, vs.SPEC_ERR_ALIGNMENT, vs.SPEC_ERR_UNSUPPORTED, vs.SPEC_ERR_WORKSPACE
NORM, READ, ATTN = target.NormRopeArgs, target.CacheReadPackedArgs, target.PrefixAttentionPackedArgs


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(vs.LIB_PATH):
        from verify_sampling_gb300 import build
        build.build()
    return vs.lib()


def _c_name(cls, field):
    """A field as C names it: those of the inner attention struct lie in `attention`."""
    inner = cls is ATTN and field not in ("k_scale", "v_scale")
    return f"attention.{field}" if inner else field


def test_every_field_sits_where_c_puts_it(tmp_path):
    structs = {"spec_norm_rope_args": NORM, "spec_cache_read_packed_args": READ, "spec_prefix_attention_packed_args": ATTN}
    lines = []
    for c, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        lines += [f'printf("%zu\\n", offsetof({c}, {_c_name(cls, f[0])}));' for f in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "spec.h"\nint main(void){' + "\n".join(lines) + "return 0;}\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    want = []
    for cls in structs.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want


def test_packed_bytes_are_the_struct():
    for call in (target._NORM_ROPE, target._READ_PACKED, target._ATTENTION_PACKED):
        values = [i + 1.5 if k is ctypes.c_float else i + 1 for i, (_, k) in enumerate(call.cls._fields_)]
        got = call.cls.from_buffer_copy(call.pack(*values))
        assert [getattr(got, f[0]) for f in call.cls._fields_] == values, call.name


def _refusals(f, cls, sizes, cases):
    """Every pointer at an address of its own (never read: the calls under test are refused)."""
    assert f(None, None) == BAD
    for change, code in cases:
        a = cls()
        for i, (name, kind) in enumerate(cls._fields_):
            if kind is ctypes.c_void_p:
                setattr(a, name, 4096 * (i + 1))
        for name, v in {**sizes, **change}.items():
            setattr(a, name, v)
        assert f(ctypes.byref(a), None) == code, change


def test_norm_rope_refuses(lib):
    sizes = dict(rows=4, Hq=8, Hk=2, D=64, rot=64, n_slots=96, eps=1e-6, scale=1.0)
    common = [({"rows": -1}, BAD), ({"Hq": -1}, BAD), ({"Hk": 1025}, BAD), ({"D": 0}, BAD), ({"rot": 63}, BAD), ({"rot": 66}, BAD),
              ({"dtype": 2}, BAD), ({"layout": 2}, BAD), ({"cache": 2}, BAD), ({"cache": -1}, BAD), ({"D": 544}, UNSUP), ({"q": None}, BAD),
              ({"q_out": None}, BAD), ({"k": None}, BAD), ({"v_cache": None}, BAD), ({"slot": None}, BAD), ({"freq": None}, BAD),
              ({"position": None}, BAD), ({"n_slots": 0}, BAD), ({"eps": -1.0}, BAD), ({"eps": float("nan")}, BAD), ({"eps": float("inf")}, BAD),
              ({"q": 4098}, ALIGN), ({"freq": 4100}, ALIGN), ({"slot": 4098}, ALIGN), ({"q_weight": 4098}, ALIGN), ({"k_weight": 4097}, ALIGN),
              ({"q": 4096, "q_out": 4096, "q_row": 512, "q_out_row": 1024}, BAD), ({"rows": 0}, vs.SPEC_OK), ({"Hq": 0, "Hk": 0}, vs.SPEC_OK)]
    _refusals(lib.spec_norm_rope_cache, NORM, sizes, common)
    _refusals(lib.spec_norm_rope_cache, NORM, {**sizes, "cache": 1, "page_size": 16}, common + [
        ({"D": 80, "rot": 80}, UNSUP), ({"page_size": 1 << 25, "n_slots": 1 << 26}, UNSUP), ({"page_size": 0}, BAD), ({"page_size": 17}, BAD), ({"k_scale": None}, BAD), ({"v_scale": None}, BAD),
        ({"k_cache": 4104}, ALIGN), ({"v_cache": 4097}, ALIGN)])


def test_cache_read_refuses(lib):
    _refusals(lib.spec_cache_read_packed, READ, dict(rows=4, Hk=2, D=64, page_size=16, n_slots=96), [
        ({"rows": -1}, BAD), ({"Hk": 0}, BAD), ({"Hk": 1025}, BAD), ({"D": 0}, BAD), ({"D": 80}, UNSUP), ({"D": 544}, UNSUP), ({"page_size": 0}, BAD),
        ({"page_size": 1 << 25, "n_slots": 1 << 26}, UNSUP), ({"page_size": 7}, BAD), ({"n_slots": -16}, BAD), ({"dtype": 2}, BAD), ({"slot": None}, BAD), ({"k_cache": None}, BAD),
        ({"v_scale": None}, BAD), ({"k_cache": 4104}, ALIGN), ({"slot": 4098}, ALIGN), ({"v": 4100}, ALIGN), ({"status": 4098}, ALIGN),
        ({"rows": 0}, vs.SPEC_OK), ({"k": None, "v": None}, vs.SPEC_OK)])


def test_attention_refuses(lib):
    need = vs.attention_packed_workspace_bytes(8, 4, 8, 64)
    assert need > 0
    for bad in ((-1, 4, 8, 64), (8, 4, 8, 288), (8, 4, 8, 80), (8, 70000, 8, 64)):
        assert vs.attention_packed_workspace_bytes(*bad) == 0
    sizes = dict(R=4, rows=8, Hq=8, Hk=2, D=64, page_size=16, n_pages=20, max_pages=4, G=2, max_prefix_pages=3, scale=0.125,
                 workspace_bytes=need)
    _refusals(lib.spec_prefix_attention_packed, ATTN, sizes, [
        ({"R": -1}, BAD), ({"R": 65536}, BAD), ({"rows": -1}, BAD), ({"Hq": 0}, BAD), ({"Hq": 7}, BAD), ({"Hk": 0}, BAD), ({"Hq": 1026}, BAD),
        ({"D": 0}, BAD), ({"D": 257}, UNSUP), ({"D": 80}, UNSUP), ({"page_size": 1 << 25, "n_pages": 2}, UNSUP), ({"dtype": 3}, BAD), ({"page_size": 0}, BAD), ({"n_pages": 0}, BAD),
        ({"max_pages": 0}, BAD), ({"G": -1}, BAD), ({"G": 5}, BAD), ({"max_prefix_pages": 0}, BAD), ({"scale": 0.0}, BAD),
        ({"scale": float("nan")}, BAD), ({"q": None}, BAD), ({"k_cache": None}, BAD), ({"out": None}, BAD), ({"row_off": None}, BAD),
        ({"kv_len": None}, BAD), ({"block_table": None}, BAD), ({"group_off": None}, BAD), ({"k_scale": None}, BAD), ({"v_scale": None}, BAD),
        ({"rows": 1 << 30, "Hq": 2}, BAD), ({"q": 4098}, ALIGN), ({"k_cache": 4104}, ALIGN), ({"lse": 4097}, ALIGN),
        ({"workspace": None}, WORK), ({"workspace_bytes": need - 1}, WORK), ({"workspace": 4096 + 128}, ALIGN),
        ({"R": 0, "G": 0}, vs.SPEC_OK), ({"rows": 0}, vs.SPEC_OK)])
