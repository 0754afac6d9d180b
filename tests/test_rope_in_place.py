"""Queries turned in place have to keep their places: other strides over the same memory would read what is written."""
import ctypes
import os

import pytest

import verify_sampling_gb300 as vs
from verify_sampling_gb300 import target


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(vs.LIB_PATH):
        from verify_sampling_gb300 import build
        build.build()
    return vs.lib()


def _args(**change):
    a = target.RopeCacheArgs()
    for i, (name, kind) in enumerate(target.RopeCacheArgs._fields_):
        if kind is ctypes.c_void_p:
            setattr(a, name, 4096 * (i + 1))  # never read: the calls are refused, or have no rows
    for name, v in {**dict(rows=4, Hq=8, Hk=2, D=64, rot=64, n_slots=100, q_row=768, q_head=64, k_row=768, k_head=64, v_row=768, v_head=64,
                           q_out_row=768, q_out_head=64), **change}.items():
        setattr(a, name, v)
    if "q_out" not in change:
        a.q_out = a.q
    return a


@pytest.mark.parametrize("change", [{"q_out_row": 512}, {"q_out_head": 96}, {"q_out_row": 512, "Hq": 1}, {"q_out_head": 96, "rows": 1},
                                    {"q_row": 0}, {"q_head": 0}])
def test_in_place_with_other_strides_is_refused(lib, change):
    assert lib.spec_rope_cache(ctypes.byref(_args(**change)), None) == vs.SPEC_ERR_INVALID_ARG


def test_strides_that_no_step_takes_do_not_matter(lib):
    """No rows: nothing is launched, whatever the strides."""
    assert lib.spec_rope_cache(ctypes.byref(_args(rows=0, q_out_row=5)), None) == vs.SPEC_OK


@pytest.mark.gpu
@pytest.mark.parametrize("rows,Hq", [(1, 4), (5, 1), (1, 1), (7, 3)])
def test_in_place_turns_alike(rows, Hq):
    """One row or one head: the stride that no step takes may differ."""
    import torch
    q = torch.randn(rows, Hq, 64, device="cuda")
    position = torch.arange(rows, dtype=torch.int32, device="cuda") + 3
    freq, _ = vs.rope_frequencies(64)
    want = vs.rope_cache(q, None, None, freq, position, None, None, None)
    out = torch.as_strided(q, q.shape, (Hq * 64 if rows > 1 else 999, 64 if Hq > 1 else 777, 1))
    assert vs.rope_cache(q, None, None, freq, position, None, None, None, q_out=out).data_ptr() == q.data_ptr()
    assert torch.equal(q, want)
    if rows > 1 and Hq > 1:
        with pytest.raises(vs.SpecError):
            vs.rope_cache(q, None, None, freq, position, None, None, None, q_out=torch.as_strided(q, q.shape, (32 * Hq, 64, 1)))
