"""No module of the tests defines a name twice: the second definition would replace the first, whose cases would never run."""
import ast
from collections import Counter
from pathlib import Path

import pytest

HERE = Path(__file__).parent
DEFS = (ast.FunctionDef, ast.AsyncFunctionDef, ast.ClassDef)


@pytest.mark.parametrize("path", sorted(HERE.glob("*.py")), ids=lambda p: p.stem)
def test_every_definition_has_a_name_of_its_own(path):
    tree = ast.parse(path.read_text())
    for scope in [tree, *(n for n in ast.walk(tree) if isinstance(n, ast.ClassDef))]:
        twice = [n for n, c in Counter(x.name for x in scope.body if isinstance(x, DEFS)).items() if c > 1]
        assert not twice, f"{path.name} defines {twice} more than once"
