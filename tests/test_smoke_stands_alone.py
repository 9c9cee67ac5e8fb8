"""CPU: what smoke() takes from tests/ is a short list that does not grow: the
entry point runs next to an older tests/ too."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# the oracle's comparison, the fp64 definitions of the first token-model operators
# and the comparison of their outputs
TAKEN = {"harness", "lm_reference", "lm_strict"}


def imported(path):
    names = set()
    for n in ast.walk(ast.parse(open(path).read())):
        if isinstance(n, ast.Import):
            names |= {a.name.split(".")[0] for a in n.names}
        elif isinstance(n, ast.ImportFrom) and n.level == 0:
            names.add(n.module.split(".")[0])
    return {n for n in names if os.path.exists(os.path.join(ROOT, "tests", n + ".py"))}


def test_the_entry_point_takes_no_other_module_of_the_tests():
    assert imported(os.path.join(ROOT, "__graft_entry__.py")) <= TAKEN
    for n in TAKEN:
        assert imported(os.path.join(ROOT, "tests", n + ".py")) <= TAKEN, n
