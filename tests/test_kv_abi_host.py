"""Host-side checks of the KV cache operators' C ABI (no GPU needed): exported symbols, struct
layouts against include/hstu_kv.h, the refusals that come before any device call, and the 64-bit
reference that the GPU tests use."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import kv_reference as R
from hstu_dense_forward_gb300 import _abi

HEADER_DIR = os.path.dirname(_abi.KV_HEADER)
OK, INVALID, UNSUPPORTED = _abi.HSTU_OK, _abi.HSTU_ERR_INVALID_ARG, _abi.HSTU_ERR_UNSUPPORTED


def test_library_exports_every_declared_symbol(built_lib):
    L = ctypes.CDLL(built_lib)
    names = _abi.declared_symbols(_abi.KV_HEADER)
    assert set(names) == {"hstu_kv_append", "hstu_kv_read", "hstu_softmax_workspace",
                          "hstu_softmax_fwd"}
    for n in names:
        assert hasattr(L, n), f"{n} declared in include/hstu_kv.h but not exported"


@pytest.mark.parametrize("struct,cls", [("hstu_kv_cache", _abi.KVCache), ("hstu_kv_rows", _abi.KVRows),
                                        ("hstu_softmax_args", _abi.SoftmaxArgs)])
def test_ctypes_mirror_matches_header(tmp_path, struct, cls):
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(
        ['#include <stddef.h>', '#include <stdio.h>', '#include "hstu_kv.h"', "int main(void) {",
         f'  printf("size %zu\\n", sizeof({struct}));'] +
        [f'  printf("{f} %zu\\n", offsetof({struct}, {f}));' for f in fields] +
        ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", HEADER_DIR, "-o", str(exe), str(src)])
    out = subprocess.check_output([str(exe)]).decode().split("\n")
    c = {k: int(v) for k, v in (line.split() for line in out if line)}
    assert c["size"] == ctypes.sizeof(cls)
    for f in fields:
        assert c[f] == getattr(cls, f).offset, f


def test_packed_structs_have_the_mirrors_layout():
    """The packs of kv_cache.py against the ctypes mirrors, field by field."""
    from hstu_dense_forward_gb300 import kv_cache as K
    for pack, cls in ((K._PACK_CACHE, _abi.KVCache), (K._PACK_ROWS, _abi.KVRows),
                      (K._PACK_ATTN, _abi.SoftmaxArgs)):
        names = [f for f, _ in cls._fields_]
        given = [0.5 if f == "alpha" else i + 1 for i, f in enumerate(names)]
        raw = pack(*given)
        assert len(raw) == ctypes.sizeof(cls)
        s = cls.from_buffer_copy(raw)
        assert [getattr(s, f) for f in names] == given


FAKE = 1 << 20  # never dereferenced: the calls fail validation first


def _cache(**kw):
    c = _abi.KVCache(dtype=_abi.HSTU_BF16, batch=2, num_heads_kv=2, head_dim=64, page_size=32,
                     index_is_int64=1, kv_cache=FAKE, num_pages=8, page_offsets=FAKE, page_ids=FAKE,
                     last_page_len=FAKE, num_page_ids=4)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _rows(**kw):
    r = _abi.KVRows(k=FAKE, v=FAKE, k_stride=128, v_stride=128, seq_offsets=FAKE, total_tokens=4,
                    dtype=_abi.HSTU_BF16)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _attn(**kw):
    a = _abi.SoftmaxArgs(q=FAKE, q_stride=256, seq_offsets=FAKE, total_tokens=4, dtype=_abi.HSTU_BF16,
                         num_heads_q=4, max_seqlen=2, max_seqlen_k=64, causal=1, alpha=0.125, out=FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHE = [
    (dict(dtype=4), INVALID), (dict(batch=-1), INVALID), (dict(batch=(1 << 20) + 1), INVALID),
    (dict(num_heads_kv=0), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=72), UNSUPPORTED),
    (dict(head_dim=272), UNSUPPORTED), (dict(page_size=64), INVALID), (dict(index_is_int64=2), INVALID),
    (dict(reserved=1), INVALID), (dict(num_pages=0), INVALID), (dict(num_page_ids=-1), INVALID),
    (dict(kv_scale=FAKE), INVALID),                                     # row scales: E4M3 only
    (dict(descale=1, k_descale=FAKE, v_descale=FAKE), INVALID),         # factors: E4M3 only
    (dict(dtype=3, descale=4, k_descale=FAKE, v_descale=FAKE), UNSUPPORTED),
    (dict(dtype=3, descale=1, k_descale=FAKE, v_descale=FAKE, kv_scale=FAKE), INVALID),
]
BAD_CACHE_POINTERS = [
    dict(kv_cache=None), dict(kv_cache=FAKE + 8), dict(page_offsets=None), dict(page_ids=None),
    dict(last_page_len=None), dict(page_offsets=FAKE + 4), dict(status=FAKE + 2),
    dict(dtype=3, descale=1), dict(dtype=3, descale=1, k_descale=FAKE),
    dict(dtype=3, k_descale=FAKE, v_descale=FAKE),
]
BAD_ROWS = [
    dict(k=None), dict(v=FAKE + 8), dict(seq_offsets=None), dict(k_stride=127), dict(v_stride=130),
    dict(total_tokens=-1), dict(total_tokens=1 << 31), dict(dtype=_abi.HSTU_F16), dict(dtype=3),
    dict(reserved=1),
]


@pytest.mark.parametrize("name", ["hstu_kv_append", "hstu_kv_read"])
def test_copies_refuse_bad_arguments(built_lib, name):
    f = getattr(_abi.lib(), name)
    by = ctypes.byref
    assert f(None, by(_rows()), None) == INVALID and f(by(_cache()), None, None) == INVALID
    for kw, want in BAD_CACHE:
        assert f(by(_cache(**kw)), by(_rows()), None) == want, kw
    for kw in BAD_CACHE_POINTERS:
        assert f(by(_cache(**kw)), by(_rows()), None) == INVALID, kw
    for kw in BAD_ROWS:
        assert f(by(_cache()), by(_rows(**kw)), None) == INVALID, kw
    assert f(by(_cache(batch=0)), by(_rows()), None) == OK          # nothing to do
    assert f(by(_cache()), by(_rows(total_tokens=0)), None) == OK


def test_attention_refuses_bad_arguments(built_lib):
    L, by = _abi.lib(), ctypes.byref
    need = ctypes.c_longlong(7)
    assert L.hstu_softmax_workspace(by(_cache()), by(_attn()), None) == INVALID
    for kw, want in BAD_CACHE:
        assert L.hstu_softmax_fwd(by(_cache(**kw)), by(_attn()), None) == want, kw
        assert L.hstu_softmax_workspace(by(_cache(**kw)), by(_attn()), by(need)) == want
        assert need.value == 0
    bad = [(dict(dtype=_abi.HSTU_F32), INVALID), (dict(dtype=3), INVALID), (dict(num_heads_q=3), INVALID),
           (dict(num_heads_q=-2), INVALID), (dict(num_heads_q=258), UNSUPPORTED),  # 129 heads share one
           (dict(max_seqlen=0), INVALID), (dict(max_seqlen_k=0), INVALID), (dict(causal=2), INVALID),
           (dict(alpha=0.0), INVALID), (dict(alpha=-1.0), INVALID), (dict(alpha=float("inf")), INVALID),
           (dict(alpha=float("nan")), INVALID), (dict(alpha=3e38), INVALID), (dict(total_tokens=-1), INVALID), (dict(reserved=1), INVALID)]
    for kw, want in bad:
        assert L.hstu_softmax_fwd(by(_cache()), by(_attn(**kw)), None) == want, kw
    for kw in (dict(batch=0),):
        assert L.hstu_softmax_fwd(by(_cache(**kw)), by(_attn()), None) == OK
    for kw in (dict(total_tokens=0), dict(num_heads_q=0)):
        assert L.hstu_softmax_fwd(by(_cache()), by(_attn(**kw)), None) == OK


def test_reference_rounding_is_e4m3():
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.1, 0.1, 20001)])
    assert np.array_equal(R.e4m3_round(x.numpy()), R.values(x.to(R.FP8)))
    assert R.e4m3_round(np.array([1e9, -np.inf]))[0] == 448
    e = R.row_exponent(np.array([[0.0], [448.0], [448.1], [1e-40], [np.inf]]))
    assert list(e) == [-100, 0, 1, -100, -100]
