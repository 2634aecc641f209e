"""Where the warps of the kernel for many rows (cache in 4 bits) turn their output
rows, read from its source.

A warp that has stored a unit's rows goes on to the next unit and writes that one's
Q, while another warp of the same 128 rows may still be turning: the scratch lies
over Q, so a warp's has to lie over its own rows alone."""
import os
import re

import pytest

from transformer_scaled_dot_02_gb300 import build as sd_build


def _source():
    return re.sub(r"//[^\n]*", "", open(os.path.join(sd_build.CSRC, "paged4_wide.cu")).read())


def _constants(text, d):
    """The integers and truth values of the kernel's configuration for heads of d columns."""
    body = text[text.index("struct WCfg"):]
    body = body[:body.index("\n};")]
    known = {"D": d}
    for name, value in re.findall(r"(k\w+) = ([^,;]+)[,;]", body):
        value = re.sub(r"(.+?) \? (.+) : (.+)", r"((\2) if (\1) else (\3))", value).replace("/", "//")
        value = re.sub(r"\b(\d+)u\b", r"\1", value)
        try:
            known[name] = eval(value, {}, known)
        except Exception:
            pass
    return known


@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
def test_a_warps_scratch_lies_over_its_own_rows(d):
    text = _source()
    c = _constants(text, d)
    stride = re.search(r"uint8_t\* turn = smem \+ sub \* C::kQBytes \+ quarter \* C::(\w+);", text).group(1)
    if not c["kTurns"]:
        return
    assert c["kQBox"] == 128 * c["kRowBytes"] and c["kTurnSlot"] == 32 * c["kTurnRow"]
    for quarter in range(4):
        first = quarter * c[stride]
        rows = (first // c["kRowBytes"], (first + c["kTurnSlot"] - 1) // c["kRowBytes"])
        assert 32 * quarter <= rows[0] and rows[1] < 32 * quarter + 32, (quarter, rows)


def test_the_heads_that_turn():
    text = _source()
    assert [d for d in (16, 32, 64, 128, 256) if _constants(text, d)["kTurns"]] == [64, 128, 256]
