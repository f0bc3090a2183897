"""The entry script as a script: what its last block calls is there by then.  Runs without a GPU."""
import ast
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_script_block_stands_behind_every_definition():
    """`python __graft_entry__.py smoke` runs the block as it is reached: a function defined
    below it does not exist yet."""
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        body = ast.parse(f.read()).body
    blocks = [n for n in body if isinstance(n, ast.If) and "__name__" in ast.unparse(n.test)]
    assert len(blocks) == 1
    late = [n.name for n in body if isinstance(n, (ast.FunctionDef, ast.ClassDef)) and n.lineno > blocks[0].lineno]
    assert not late, late
