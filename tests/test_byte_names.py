"""The 8-bit calls go by two names, and the measured cases call names that exist."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from paged_kv_cache_req_gb300 import build
    build.build()
    from paged_kv_cache_req_gb300 import _binding
    return _binding


def test_both_names_are_one_function(B):
    for name in [n for n in dir(B) if n.startswith("pkv_byte_")] + ["make_byte_args"]:
        assert getattr(B, name.replace("_byte_", "_q8_")) is getattr(B, name), name


@pytest.mark.parametrize("name", ["operators.py", "more_operators.py"])
def test_measured_cases_call_what_there_is(B, name):
    text = open(os.path.join(ROOT, "perf", name)).read()
    called = set(re.findall(r"\bB\.(\w+)", text))
    assert called
    for x in called:
        assert hasattr(B, x), x


def test_the_names_that_the_first_cases_call(B):
    for x in ("make_q8_args", "pkv_q8_store", "pkv_q8_store_workspace_size", "pkv_q8_gather", "pkv_q8_decode", "pkv_q8_extend",
              "pkv_q8_weights", "pkv_q8_decode_workspace_size", "pkv_q8_extend_workspace_size", "pkv_q8_weights_workspace_size"):
        assert callable(getattr(B, x)), x
