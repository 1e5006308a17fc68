"""Inline assembly names the registers that it writes by hand (CPU)."""
import pathlib
import re

import linear_attention_speculative_amd as kda

CSRC = pathlib.Path(kda.__file__).parent / "csrc"


def statements():
    for path in sorted(CSRC.glob("*.h*")):
        for m in re.finditer(r"asm volatile\((.*?)\);", path.read_text(),
                             re.S):
            yield path.name, m.group(1)


def test_m0_is_declared_where_it_is_written():
    found = [(name, text) for name, text in statements()
             if re.search(r"s_mov_b32 m0,", text)]
    assert len(found) >= 3
    for name, text in found:
        clobbers = text.rsplit(":", 1)[1]
        assert '"m0"' in clobbers and '"memory"' in clobbers, (name, text)
