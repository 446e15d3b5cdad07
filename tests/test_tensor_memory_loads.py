"""Loads from tensor memory are asynchronous: what they bring may be used behind a wait only.

An instruction on registers is not kept behind a wait that does not name them, so each wait names what was
loaded, and each load's destination is named by a wait before anything else.  Read from the sources: the
compiler's present order of instructions does not show it."""
import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "speculative_decoding_verification_sdcp_gb300", "csrc", "*.cu*")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_what_a_load_brings_is_named_by_a_wait(path):
    text = open(path).read()
    for wait in re.finditer(r"tcgen05\.wait::ld[^;]*;\"(?P<operands>.*?)\);\n", text, re.S):
        assert '"+f"' in wait["operands"]
    for load in re.finditer(r"tmem_ld\d+\([^;{]*\b(?P<into>\w+)\);", text):
        use = re.search(r"[^\n]*\b%s\b" % load["into"], text[load.end():])
        assert use and use[0].strip().endswith("tmem_loaded(" + load["into"]), load[0]
