"""The entry script at the repository's root, without a GPU."""
import ast
import os


def test_the_entry_script_defines_all_before_it_runs():
    """`python __graft_entry__.py smoke`: what smoke() calls stands above the line that calls it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "__graft_entry__.py")) as f:
        body = ast.parse(f.read()).body
    runs = [i for i, node in enumerate(body)
            if isinstance(node, ast.If) and "__name__" in ast.dump(node.test)]
    assert runs == [len(body) - 1]
