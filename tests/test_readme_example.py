"""The usage example: its calls bind to the functions as they are, and the ones
that turn positions take the magnitude that goes with the frequencies."""
import ast
import inspect
import os
import re

import gated_delta_rule_49_amd as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def calls():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    for node in ast.walk(ast.parse("\n".join(blocks))):
        if isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute) and isinstance(node.func.value, ast.Name) and node.func.value.id == "kda":
            yield node.func.attr, inspect.signature(getattr(kda, node.func.attr)).bind(*node.args, **{k.arg: k.value for k in node.keywords}).arguments


def test_calls_bind():
    names = {name for name, _ in calls()}
    assert {"prefill", "latent_append", "rotary", "rotary_backward", "latent_prefill", "latent_backward", "latent_decode"} <= names


def test_positions_are_turned_with_their_magnitude():
    for name, given in calls():
        if "freqs" in given:
            assert isinstance(given.get("magnitude"), ast.Name) and given["magnitude"].id == "magnitude", f"{name} without the frequencies' magnitude"


def test_gradients_are_turned_back_as_the_forward_turned():
    turned = [g for name, g in calls() if name == "rotary"]
    for given in (g for name, g in calls() if name == "rotary_backward"):
        same = {k: ast.dump(v) for k, v in given.items() if k not in ("x", "d_out")}
        assert any(same == {k: ast.dump(v) for k, v in g.items() if k != "x"} for g in turned)
