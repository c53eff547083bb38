"""__graft_entry__.py run as a script: every name that its functions use is there by the
time the last block runs them."""
import ast
import os
import sys

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "__graft_entry__.py")


def _script():
    """The file with each function's body replaced by a look at the file's own names in it,
    and a call of those that are functions."""
    tree = ast.parse(open(PATH).read())
    functions = {n.name for n in tree.body if isinstance(n, ast.FunctionDef)}
    for n in tree.body:
        if isinstance(n, ast.FunctionDef):
            used = {x.id for x in ast.walk(n) if isinstance(x, ast.Name) and isinstance(x.ctx, ast.Load)}
            lines = [f"ran.append({n.name!r})"] + [f"{x}()" for x in sorted(used & functions)]
            n.body = ast.parse("\n".join(lines)).body
    return compile(ast.fix_missing_locations(tree), PATH, "exec"), functions


@pytest.mark.parametrize("args,wanted", [([], {"build"}), (["smoke"], None)])
def test_the_script_reaches_all_that_it_calls(monkeypatch, args, wanted):
    code, functions = _script()
    assert {"build", "smoke", "_smoke_packed", "_smoke_paged"} <= functions
    monkeypatch.setattr(sys, "argv", [PATH] + args)
    monkeypatch.setattr(sys, "path", list(sys.path))
    ran = []
    exec(code, {"__name__": "__main__", "__file__": PATH, "ran": ran})
    assert set(ran) == (functions if wanted is None else wanted)
