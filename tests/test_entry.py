"""The build and smoke entry points as a script."""
import ast
import os
import subprocess
import sys

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "__graft_entry__.py")


def test_script_part_stands_behind_every_definition():
    with open(PATH) as f:
        body = ast.parse(f.read()).body
    at = [i for i, node in enumerate(body) if isinstance(node, ast.If) and "__main__" in ast.unparse(node.test)]
    assert at == [len(body) - 1]


def test_script_builds():
    assert subprocess.run([sys.executable, PATH], timeout=900).returncode == 0


@pytest.mark.gpu
def test_script_runs_the_smoke_step():
    r = subprocess.run([sys.executable, PATH, "smoke"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    assert "smoke ok" in r.stdout
