"""Host-side checks of the eviction operators' C ABI (no GPU needed): exported symbols, struct
layouts against include/hstu_evict.h, the refusals that come before any device call, those of the
4-bit cache, and the 64-bit references that the GPU tests use."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import evict_reference as E
import kv4_reference as R4
from hstu_dense_forward_gb300 import _abi

HEADER_DIR = os.path.dirname(_abi.EVICT_HEADER)
OK, INVALID, UNSUPPORTED = _abi.HSTU_OK, _abi.HSTU_ERR_INVALID_ARG, _abi.HSTU_ERR_UNSUPPORTED
FAKE = 1 << 20  # never dereferenced: the calls fail validation first


def test_library_exports_every_declared_symbol(built_lib):
    L = ctypes.CDLL(built_lib)
    names = _abi.declared_symbols(_abi.EVICT_HEADER)
    assert set(names) == {"hstu_kv_weights", "hstu_kv_select", "hstu_compact_workspace",
                          "hstu_kv_compact"}
    for n in names:
        assert hasattr(L, n), f"{n} declared in include/hstu_evict.h but not exported"


@pytest.mark.parametrize("struct,cls", [("hstu_weights_args", _abi.WeightsArgs),
                                        ("hstu_select_args", _abi.SelectArgs),
                                        ("hstu_compact_args", _abi.CompactArgs),
                                        ("hstu_kv_cache", _abi.KVCache)])
def test_ctypes_mirror_matches_header(tmp_path, struct, cls):
    fields = [f for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(
        ['#include <stddef.h>', '#include <stdio.h>', '#include "hstu_evict.h"', "int main(void) {",
         f'  printf("size %zu\\n", sizeof({struct}));'] +
        [f'  printf("{f} %zu\\n", offsetof({struct}, {f}));' for f in fields] +
        ['  printf("fp4 %d\\n", HSTU_FP4_E2M1);', "  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", HEADER_DIR, "-o", str(exe), str(src)])
    out = subprocess.check_output([str(exe)]).decode().split("\n")
    c = {k: int(v) for k, v in (line.split() for line in out if line)}
    assert c["size"] == ctypes.sizeof(cls) and c["fp4"] == _abi.HSTU_FP4_E2M1
    for f in fields:
        assert c[f] == getattr(cls, f).offset, f


def test_packed_structs_have_the_mirrors_layout():
    from hstu_dense_forward_gb300 import evict as V
    for pack, cls in ((V._PACK_WEIGHTS, _abi.WeightsArgs), (V._PACK_SELECT, _abi.SelectArgs),
                      (V._PACK_COMPACT, _abi.CompactArgs)):
        names = [f for f, _ in cls._fields_]
        given = [0.5 if f == "alpha" else i + 1 for i, f in enumerate(names)]
        raw = pack(*given)
        assert len(raw) == ctypes.sizeof(cls)
        s = cls.from_buffer_copy(raw)
        assert [getattr(s, f) for f in names] == given


def _set(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _cache(**kw):
    return _set(_abi.KVCache(dtype=_abi.HSTU_BF16, batch=2, num_heads_kv=2, head_dim=64, page_size=32,
                             index_is_int64=1, kv_cache=FAKE, num_pages=8, page_offsets=FAKE, page_ids=FAKE,
                             last_page_len=FAKE, num_page_ids=4), kw)


def _fp4(**kw):
    return _cache(**{**dict(dtype=_abi.HSTU_FP4_E2M1, kv_scale=FAKE, kv_group_scale=FAKE), **kw})


def _weights(**kw):
    return _set(_abi.WeightsArgs(q=FAKE, q_stride=256, seq_offsets=FAKE, total_tokens=4, dtype=_abi.HSTU_BF16,
                                 num_heads_q=4, max_seqlen=2, max_seqlen_k=64, causal=1, alpha=0.125, lse=FAKE,
                                 weights=FAKE, accumulate=1), kw)


def _select(**kw):
    return _set(_abi.SelectArgs(batch=2, num_heads_kv=2, page_size=32, index_is_int64=1, num_pages=8,
                                page_offsets=FAKE, page_ids=FAKE, last_page_len=FAKE, num_page_ids=4, weights=FAKE,
                                budget=16, recent=4, max_seqlen_k=64, kept=FAKE, new_page_offsets=2 * FAKE,
                                new_page_ids=2 * FAKE, new_last_page_len=2 * FAKE), kw)


def _compact(**kw):
    return _set(_abi.CompactArgs(kept=FAKE, budget=16, max_seqlen_k=64), kw)


def test_weights_refuse_bad_arguments(built_lib):
    f, by = _abi.lib().hstu_kv_weights, ctypes.byref
    assert f(None, by(_weights()), None) == INVALID and f(by(_cache()), None, None) == INVALID
    bad = [(dict(dtype=_abi.HSTU_F32), INVALID), (dict(dtype=3), INVALID), (dict(num_heads_q=3), INVALID),
           (dict(num_heads_q=-2), INVALID), (dict(num_heads_q=258), UNSUPPORTED), (dict(max_seqlen=0), INVALID),
           (dict(max_seqlen=(1 << 24) + 1), INVALID), (dict(max_seqlen_k=0), INVALID), (dict(causal=2), INVALID),
           (dict(alpha=0.0), INVALID), (dict(alpha=float("nan")), INVALID), (dict(alpha=3e38), INVALID),
           (dict(total_tokens=-1), INVALID), (dict(total_tokens=1 << 31), INVALID), (dict(reserved=1), INVALID),
           (dict(accumulate=2), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID),
           (dict(lse=None), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(weights=None), INVALID),
           (dict(weights=FAKE + 4), INVALID), (dict(seq_offsets=None), INVALID), (dict(q_stride=255), INVALID),
           (dict(q_stride=260), INVALID)]
    for kw, want in bad:
        assert f(by(_cache()), by(_weights(**kw)), None) == want, kw
    for kw in (dict(page_ids=None), dict(kv_cache=FAKE + 8), dict(page_size=64), dict(dtype=4)):
        assert f(by(_cache(**kw)), by(_weights()), None) == INVALID, kw
    assert f(by(_cache(batch=0)), by(_weights()), None) == OK
    assert f(by(_cache()), by(_weights(total_tokens=0, q=None, lse=None)), None) == OK


def test_select_refuses_bad_arguments(built_lib):
    f, by = _abi.lib().hstu_kv_select, ctypes.byref
    assert f(None, None) == INVALID
    for kw in (dict(batch=-1), dict(num_heads_kv=0), dict(page_size=64), dict(index_is_int64=2), dict(num_pages=0),
               dict(num_page_ids=-1), dict(budget=0), dict(budget=(1 << 30) + 1), dict(recent=-1),
               dict(max_seqlen_k=0), dict(reserved=1), dict(page_offsets=None), dict(page_ids=None),
               dict(last_page_len=None), dict(weights=None), dict(weights=FAKE + 4), dict(kept=None),
               dict(kept=FAKE + 2), dict(new_page_offsets=None), dict(new_page_ids=None),
               dict(new_last_page_len=None), dict(new_page_offsets=FAKE), dict(new_page_ids=FAKE),
               dict(new_last_page_len=FAKE), dict(page_offsets=FAKE + 4), dict(status=FAKE + 1)):
        assert f(by(_select(**kw)), None) == INVALID, kw
    assert f(by(_select(batch=0)), None) == OK


def test_compact_refuses_bad_arguments(built_lib):
    L, by = _abi.lib(), ctypes.byref
    need = ctypes.c_longlong(7)
    assert L.hstu_compact_workspace(by(_cache()), by(_compact()), None) == INVALID
    assert L.hstu_kv_compact(None, by(_compact()), None) == INVALID
    assert L.hstu_kv_compact(by(_cache()), None, None) == INVALID
    for kw in (dict(budget=0), dict(max_seqlen_k=0), dict(reserved=1)):
        assert L.hstu_kv_compact(by(_cache()), by(_compact(**kw)), None) == INVALID, kw
        assert L.hstu_compact_workspace(by(_cache()), by(_compact(**kw)), by(need)) == INVALID
        assert need.value == 0
    for kw in (dict(kept=None), dict(kept=FAKE + 2), dict(weights=FAKE + 4)):
        assert L.hstu_kv_compact(by(_cache()), by(_compact(**kw)), None) == INVALID, kw
    for kw in (dict(kv_cache=None), dict(page_ids=None), dict(page_size=64)):
        assert L.hstu_kv_compact(by(_cache(**kw)), by(_compact()), None) == INVALID, kw
    assert L.hstu_kv_compact(by(_cache(batch=0)), by(_compact()), None) == OK


def test_four_bit_caches_refuse_bad_arguments(built_lib):
    L, by = _abi.lib(), ctypes.byref
    rows = _abi.KVRows(k=FAKE, v=FAKE + 4096, k_stride=128, v_stride=128, seq_offsets=FAKE, total_tokens=4,
                       dtype=_abi.HSTU_BF16)
    attn = _abi.SoftmaxArgs(q=FAKE, q_stride=256, seq_offsets=FAKE, total_tokens=4, dtype=_abi.HSTU_BF16,
                            num_heads_q=4, max_seqlen=2, max_seqlen_k=64, causal=1, alpha=0.125, out=FAKE)
    for kw, want in ((dict(kv_scale=None), INVALID), (dict(kv_group_scale=None), INVALID),
                     (dict(kv_group_scale=FAKE + 8), INVALID), (dict(kv_scale=FAKE + 8), INVALID),
                     (dict(head_dim=48), UNSUPPORTED), (dict(head_dim=288), UNSUPPORTED),
                     (dict(descale=1, k_descale=FAKE, v_descale=FAKE), INVALID),
                     (dict(descale=1), INVALID), (dict(k_descale=FAKE), INVALID)):
        assert L.hstu_kv_append(by(_fp4(**kw)), by(rows), None) == want, kw
        assert L.hstu_kv_read(by(_fp4(**kw)), by(rows), None) == want, kw
        if want == UNSUPPORTED or "descale" in kw:  # (pointers: after the device is asked)
            assert L.hstu_softmax_fwd(by(_fp4(**kw)), by(attn), None) == want, kw
        assert L.hstu_kv_weights(by(_fp4(**kw)), by(_weights()), None) == want, kw
        assert L.hstu_kv_compact(by(_fp4(**kw)), by(_compact()), None) == want, kw
    # sizes alone decide on workspaces
    need = ctypes.c_longlong(7)
    assert L.hstu_softmax_workspace(by(_fp4(batch=0, kv_scale=None, kv_group_scale=None)), by(attn), by(need)) == OK


def test_append_with_weights_refuses_bad_arguments(built_lib):
    """hstu_kv_rows.weights counts where hstu_kv_rows.reserved says that the struct has it."""
    L, by = _abi.lib(), ctypes.byref

    def rows(**kw):
        return _set(_abi.KVRows(k=FAKE, v=2 * FAKE, k_stride=128, v_stride=128, seq_offsets=FAKE, total_tokens=4,
                                dtype=_abi.HSTU_BF16, reserved=_abi.HSTU_ROWS_WEIGHTS, weights=FAKE), kw)

    for kw in (dict(weights=FAKE + 4), dict(reserved=1), dict(reserved=3), dict(k=None)):
        assert L.hstu_kv_append(by(_cache()), by(rows(**kw)), None) == INVALID, kw
    assert L.hstu_kv_read(by(_cache()), by(rows()), None) == INVALID  # no call to write weights
    assert L.hstu_kv_append(by(_cache()), by(rows(total_tokens=0)), None) == OK


def test_references():
    m = np.array([0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 3.5, 5.0, 5.01, 100.0, -0.3])
    assert list(R4.E2M1[R4.e2m1_code(m)]) == [0, 0.5, 1, 0.5, 1, 1.5, 2, 2, 4, 4, 6, 6, -0.5]
    code, factor, e = R4.quantise(np.array([[2688.0] + [6.0] * 15 + [0.0] * 16, [1e-40] * 32]))
    assert factor[0, 0] == 448 and factor[0, 1] == 0 and list(e) == [0, -100] and not code[1].any()
    w = np.array([3.0, 1.0, 3.0, np.nan, 0.0, 3.0, 2.0, -1.0])
    assert E.select(w, 4, 0) == [0, 2, 5, 6] and E.select(w, 3, 0) == [0, 2, 5]
    assert E.select(w, 2, 0) == [0, 2] and E.select(w, 3, 2) == [0, 6, 7] and E.select(w, 9, 1) == list(range(8))
    assert E.select(w, 1, 5) == [7] and E.select(w, 7, 0) == [0, 1, 2, 4, 5, 6, 7] and E.select(w[:0], 3, 1) == []
