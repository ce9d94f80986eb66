"""What the calls of the package's top level need is there too."""

import ast
import os

import collective_matmul_decomposition_gb300 as package
from collective_matmul_decomposition_gb300 import cm


def test_workspace_sizes_are_exported():
    for name in ("linear_wgrad_workspace_size", "layer_norm_backward_workspace_size"):
        assert getattr(package, name) is getattr(cm, name)


def test_every_binding_is_exported():
    """Each module-level function of the binding that calls the library, but those named otherwise at the top level."""
    with open(os.path.join(os.path.dirname(cm.__file__), "cm.py")) as f:
        tree = ast.parse(f.read())
    new = [n.name for n in tree.body if isinstance(n, ast.FunctionDef)
           and n.name.startswith(("cm_linear", "cm_layer_norm", "cm_adamw", "linear_", "layer_norm_"))]
    assert len(new) >= 9
    for name in new:
        assert getattr(package, name) is getattr(cm, name), name
