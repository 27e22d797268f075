"""Every file that checks indexes in the checks build has a word of its own there, and
moe_checks_read collects it.  Host only."""
import glob
import os
import re

from moe_expert_layer_softmax_gb300 import _build


def test_words_are_registered_and_read():
    with open(os.path.join(_build.CSRC, "api.cu")) as f:
        read = set(re.findall(r"check_word_(\w+)\(\)", f.read()))
    seen = set()
    for path in glob.glob(os.path.join(_build.CSRC, "*.cu")):
        with open(path) as f:
            text = f.read()
        words = set(re.findall(r"MOE_CHECK_WORD_ACCESSOR\((\w+)\)", text))
        assert words or not re.search(r"MOE_CHECKED\(|MOE_CHECK_OK\(", text), path
        seen |= words
    assert seen == read and "few" in seen
