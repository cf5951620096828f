"""The repository's entry file run as a script: the block that runs it comes behind all that it calls."""
import ast
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["__graft_entry__.py", "bench.py", "examples/rollout_and_update.py",
                                  "examples/tied_policy_step.py"])
def test_nothing_is_defined_behind_the_main_block(name):
    body = ast.parse(open(os.path.join(ROOT, name)).read()).body
    blocks = [i for i, node in enumerate(body) if isinstance(node, ast.If) and "__name__" in ast.dump(node.test)]
    assert blocks == [len(body) - 1], name
