"""Inline assembly of the kernels names what it changes: a statement that steps M0 with a
scalar add also sets SCC, where the compiler may be keeping a loop's condition or a carry."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# scalar instructions that write SCC
SETS_SCC = re.compile(r"\bs_(add|sub|addc|subb|addk|and|or|xor|andn2|orn2|nand|nor|xnor|not|lshl\w*|lshr|ashr|bfe|abs|absdiff|"
                      r"min|max|cmp\w*|cmpk\w*|bitcmp\w*|wqm|quadmask|bcnt\w*)_\w+")


def statements(text):
    for m in re.finditer(r"\basm\s+(?:volatile\s*)?\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.start():i]


def test_statements_that_set_scc_say_so():
    seen = 0
    for path in sorted(glob.glob(os.path.join(ROOT, "dense_blas3_gemm_amd", "csrc", "*"))):
        for s in statements(open(path).read()):
            if SETS_SCC.search(s):
                seen += 1
                assert '"scc"' in s, f"{path}: {s}"
    assert seen >= 3
