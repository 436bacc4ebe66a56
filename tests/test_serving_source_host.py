"""The CPU model of the few-token kernels' addressing (test_serving_addressing.py) against the source: its
constants are the kernels', and the int4 words of a panel end with the matrix."""
import os
import re

import numpy as np
import pytest

from _util import ROOT
import test_serving_addressing as model

CSRC = os.path.join(ROOT, "mixture_experts_routed_route_amd", "csrc")


def source(name):
    return open(os.path.join(CSRC, name)).read()


def test_model_has_the_kernels_constants():
    text = source("few_tokens.h") + source("few_tokens.hip")

    def constant(name):
        found = re.findall(rf"constexpr (?:int|uint16_t) {name} = ([^;]+);", text)
        assert len(found) == 1, name
        return eval(found[0], {}, {"kMaxE": model.MAX_E, "kFewMaxHidden": 65536})   # sums of the constants
    assert constant("kFewTokens") == model.TOKENS and constant("kFewTopK") == model.TOPK
    assert constant("kMaxE") == model.MAX_E and constant("kGroups") == model.GROUPS
    assert constant("kNoToken") == model.NO_TOKEN
    assert (constant("kFewDownGrid"), constant("kFewMaxSplits"), constant("kFewMaxHidden")) == (256, 16, 65536)
    # LDS left for x, waves and granules of the streams
    assert f"return {model.LDS} - 256 - static_cast<int>(sizeof(Routed)) - nw * cpl * 1024;" in text
    assert "return src != kPair ? 4 : steps == 4 ? 2 : 3;" in text and "NW = 4 * min_waves(STEPS, SRC)" in text
    assert "Rows<KIND, 2, KIND != kBf16 ? 2 : SRC == kTile ? 4 : 3, SRC>" in text
    for group, steps, row in ((32, 1, 1), (64, 2, 2), (128, 4, 2), (256, 4, 2)):
        assert re.search(rf"case {group}:(?:\s*case \d+:)*\s*return launch_kind<kInt4, {steps}, {row}>", text), group
        assert model.shape("int4", group, "tile")[1] == 32 * steps and model.shape("int4", group, "row")[1] == 32 * row


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("T,E,k,H,I", model.CASES)
def test_int4_words_end_with_the_matrix(group, T, E, k, H, I):
    """The last word that a panel's last granule reads is the last of the expert's matrix, in both launches."""
    step = max(64, group)
    H, I = -(-H // step) * step, -(-I // step) * step
    for src, N, K in (("tile", I, H), ("row", I, H), ("pair", H, I)):
        cols, unit, _ = model.shape("int4", group, src)
        grans, panels = K // unit, -(-N // cols)
        last = ((grans - 1) * (unit // 8) + (unit // 32 - 1) * 4 + 3) * N + (panels - 1) * cols + 64
        assert grans * unit == K and last == K // 8 * N
