"""How the kernel for many rows (cache in 4 bits) reads what the caller's kernels
wrote, from its source.

It begins beside the kernel for the other sequences and waits for that one at its end
only.  That one's blocks have waited for all kernels before, so queries, starts,
lengths, the table and the pages are in L2; a line that an SM's L1 still holds from an
earlier call could be older, and no wait of this kernel's own puts it away."""
import os
import re

from transformer_scaled_dot_02_gb300 import build as sd_build


def test_inputs_are_read_past_l1():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(sd_build.CSRC, "paged4_wide.cu")).read())
    kernel = text[text.index("__global__"):]
    wait = [m.start() for m in re.finditer(r"griddep_wait\(\)", kernel)]
    assert wait and kernel.index("find_place(plan") < wait[-1]
    for name in ("p.q_starts", "p.kv_lengths"):
        uses = re.findall(r"(\S{0,8})" + re.escape(name) + r"\b", text)
        assert uses and all(u.endswith("__ldcg(") for u in uses), (name, uses)
    # the table through `pages`, queries through `src`; pages by cp.async.cg
    assert re.findall(r"(\S{0,7})pages \+ \(key", kernel) == ["__ldcg("] and not re.search(r"\bpages\[", kernel)
    assert "__ldcg(reinterpret_cast<const uint4*>(src)" in kernel and not re.search(r"\(src\)\[", kernel)
    assert "cp.async.ca" not in text and "cp.async.cg.shared.global" in text
