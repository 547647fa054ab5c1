"""The smoke check reports the status that it read."""
import ast
import inspect

import pytest

import __graft_entry__ as entry
import submanifold_sparse_convolution_gb300 as sc
from submanifold_sparse_convolution_gb300 import build as build_mod


def test_smoke_reads_each_status_once():
    """rows_status clears the word that it reports: a second reading says 'ok'."""
    calls = [n.func.attr for n in ast.walk(ast.parse(inspect.getsource(entry.smoke)))
             if isinstance(n, ast.Call) and isinstance(n.func, ast.Attribute)]
    assert calls.count("rows_status") == 1 and calls.count("map_status") == 1


def test_a_status_is_named_in_the_error():
    build_mod.build()
    entry._require_ok(0, sc.status_string)
    with pytest.raises(RuntimeError, match="kernel wait timed out"):
        entry._require_ok(-8, sc.status_string)
