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
