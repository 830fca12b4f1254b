"""__graft_entry__.py run as a script has all that it has when it is imported."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_script_runs_after_its_functions_are_defined():
    body = ast.parse(open(os.path.join(ROOT, "__graft_entry__.py")).read()).body
    runs = [i for i, x in enumerate(body) if isinstance(x, ast.If) and "__main__" in ast.unparse(x.test)]
    assert runs == [len(body) - 1]
