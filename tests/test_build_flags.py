"""How the library's sources are compiled (bit_recurrent_state_amd/build.py)."""
import importlib.util
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "bit_recurrent_state_amd")


def _build():
    spec = importlib.util.spec_from_file_location("_pace_build_flags", os.path.join(PACKAGE, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_sources_with_defined_results_for_nan_honour_it():
    """pace_cache.h says what its calls make of NaN, so no source of theirs may be compiled as if
    there were none: comparisons and maxima with one would be the compiler's choice."""
    b = _build()
    for src in b.SOURCES:
        text = open(os.path.join(PACKAGE, "csrc", src)).read()
        if re.search(r'#include "pace_(cache_internal|attention)\.h"', text):
            assert src in b.HONOR_NANS, src
    assert b.HONOR_NANS <= set(b.SOURCES)
    assert not any("nans" in f or "finite-math" in f or "fast-math" in f for f in b.COMMON)
