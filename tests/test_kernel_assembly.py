"""What the kernels' assembly blocks change and the compiler does not see: m0 and
the scalar condition code are declared where a block writes them, and the
execution mask is put back from what it was, not from what it is taken to be."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_paged_cache_amd", "csrc")
# scalar instructions that leave a condition code (moves and waits do not)
SETS_SCC = re.compile(r"\bs_(?:and|or|xor|andn2|add|sub|lshl|lshr|cmp|not|bcnt)\w*")


def blocks():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            body = text[m.end():i - 1]
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', re.split(r'"\s*:', body, maxsplit=1)[0] + '"'))
            yield f"{os.path.basename(path)}:{text.count(chr(10), 0, m.start()) + 1}", code.replace("\\n\\t", "\n"), body


BLOCKS = list(blocks())


def test_blocks_are_found():
    assert sum("global_load_lds" in code for _, code, _ in BLOCKS) >= 5
    assert sum("mfma" in code for _, code, _ in BLOCKS) >= 1


@pytest.mark.parametrize("where,code,body", BLOCKS, ids=[b[0] for b in BLOCKS])
def test_a_block_declares_what_it_writes(where, code, body):
    clobbers = body.rsplit(":", 1)[1]
    if re.search(r"\bs_mov_b32 m0\b", code):
        assert '"m0"' in clobbers, where
    if SETS_SCC.search(code):
        assert '"scc"' in clobbers, where
    if re.search(r"\bexec\b", code) or "saveexec" in code:
        saved = re.search(r"s_and_saveexec_b64 (%\w+)", code)
        assert saved, f"{where}: the mask is not saved"
        for source in re.findall(r"s_mov_b64 exec, (\S+)", code):
            assert source == saved.group(1), f"{where}: the mask is set to {source}"
        assert code.count("saveexec") == code.count("s_mov_b64 exec,"), where
