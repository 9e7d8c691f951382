"""Host-side checks of the KV cache operators' Python entry points (no GPU needed)."""
import ast
import inspect
import os
import re

import hstu_dense_forward_gb300 as hstu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _documented_calls():
    """Calls of the package's functions in the indented paragraphs of README.md."""
    text = open(os.path.join(ROOT, "README.md")).read()
    for block in re.findall(r"(?:^    .*\n)+", text, flags=re.M):
        code = "\n".join(line[4:] for line in block.split("\n"))
        try:
            tree = ast.parse(code)
        except SyntaxError:  # shell commands
            continue
        for node in ast.walk(tree):
            if isinstance(node, ast.Call) and isinstance(node.func, ast.Name) and \
                    node.func.id in hstu.__all__:
                yield node


def test_documented_calls_pass_what_the_parameters_are_called():
    seen = set()
    for call in _documented_calls():
        f = getattr(hstu, call.func.id)
        seen.add(call.func.id)
        positional = [p.name for p in inspect.signature(f).parameters.values()
                      if p.kind is p.POSITIONAL_OR_KEYWORD]
        given = [a.id for a in call.args]
        assert given == positional[:len(given)], call.func.id
        names = set(inspect.signature(f).parameters)
        assert {k.arg for k in call.keywords if k.arg} <= names, call.func.id
    assert {"hstu_fwd", "hstu_kv_append", "hstu_softmax_fwd"} <= seen


def test_read_refuses_one_place_for_keys_and_values(built_lib):
    """The library's check (no device call before it): k and v of a read are written."""
    import ctypes
    from hstu_dense_forward_gb300 import _abi
    at = 1 << 20  # never dereferenced
    cache = _abi.KVCache(dtype=_abi.HSTU_BF16, batch=2, num_heads_kv=2, head_dim=64, page_size=32,
                         index_is_int64=1, kv_cache=at, num_pages=8, page_offsets=at, page_ids=at,
                         last_page_len=at, num_page_ids=4)
    rows = _abi.KVRows(k=at, v=at, k_stride=128, v_stride=128, seq_offsets=at, total_tokens=4,
                       dtype=_abi.HSTU_BF16)
    assert _abi.lib().hstu_kv_read(ctypes.byref(cache), ctypes.byref(rows), None) == \
        _abi.HSTU_ERR_INVALID_ARG
