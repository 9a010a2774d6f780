"""The calls that the README shows can be made: every api function in its Python blocks exists and
takes the arguments as they are written there."""

import ast
import inspect
import os
import re

from bitwise_consistent_linear_amd import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_fit_their_functions():
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    calls = [node for block in blocks for node in ast.walk(ast.parse(block))
             if isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute)
             and isinstance(node.func.value, ast.Name) and node.func.value.id == "api"]
    assert len(calls) >= 15
    for call in calls:
        fn = getattr(api, call.func.attr)
        if any(isinstance(a, ast.Starred) for a in call.args) or any(
                k.arg is None for k in call.keywords):
            continue
        inspect.signature(fn).bind(*call.args, **{k.arg: k.value for k in call.keywords})
