"""How a gated or 8-bit integer call is run: the library's own choice (pure host code)."""
import ctypes
from collections import namedtuple

import dense_blas3_gemm_amd as d

OPS = {"i8": 0, "gated": 1, "dgated": 2}
KINDS = {"bf16": 0, "e4m3": 1, "i8": 2}
Launch = namedtuple("Launch", "kernel splits rows cols")


def plan(op, kind, tB, M, N, K, sums=False, pad=0, cus=256):
    """The launches of a call (without those that add up), each Launch(kernel, splits, rows, cols)."""
    fn = d.load_library().dbgemm_gated_plan
    i64 = ctypes.c_int64
    fn.argtypes = [ctypes.c_int] * 3 + [i64] * 6 + [ctypes.c_int] * 2 + [ctypes.c_char_p, ctypes.c_size_t]
    text = ctypes.create_string_buffer(1 << 16)
    ldb = (K if tB else N) + pad
    assert fn(OPS[op], KINDS[kind], tB, M, N, K, K + pad, ldb, ldb, int(sums), cus, text, len(text)) == 0
    out = []
    for one in text.value.decode().split("; "):
        kernel, size = one.split(" ")
        kernel, _, splits = kernel.partition("+sk")
        rows, cols = size.split("x")
        out.append(Launch(kernel, int(splits or 1), int(rows), int(cols)))
    return out


# (operator, operands, B [N][K])
FORMS = [(op, kind, tB) for op, kind in (("gated", "bf16"), ("gated", "e4m3"), ("gated", "i8"), ("dgated", "bf16"),
                                         ("dgated", "e4m3"), ("i8", "i8")) for tB in (0, 1)]

# Products that between them are run on every kernel, in every form: rows and columns of no whole tiles, K of
# no whole K tile.
SHAPES = [(1, 16, 16), (3, 4272, 432), (7, 9104, 176), (8, 8720, 3888), (15, 12496, 1328), (18, 4144, 144),
          (19, 16, 16), (23, 8288, 1312), (23, 8736, 2400), (25, 4112, 736), (25, 8560, 304), (35, 16, 16),
          (36, 4176, 720), (46, 4176, 1856), (100, 32, 2992), (524, 13600, 16), (3310, 672, 9584), (5755, 1424, 4512),
          (6631, 80, 9840), (7503, 2224, 48), (7707, 2080, 32), (10831, 1488, 8528), (11900, 1392, 4176),
          (15077, 1104, 2416), (16732, 80, 176), (16914, 144, 16), (16997, 48, 32), (17034, 48, 10480),
          (17108, 144, 9024), (19226, 112, 8944)]
PAD = 16  # of every operand's rows


def form_plan(form, shape):
    return plan(*form, *shape, sums=form[0] == "dgated", pad=PAD)


def instances(form, shape):
    """The kernels that a product is run on, split or not, few rows by 16, 32 or 64 of them; and where it is run
    in two launches, along what and whether the second one is split."""
    p = form_plan(form, shape)
    rows = 16 if shape[0] <= 16 else 32 if shape[0] <= 32 else 64
    out = {(x.kernel, rows) if x.kernel.startswith("few_rows") else (x.kernel, "split" if x.splits > 1 else "whole")
           for x in p}
    if len(p) == 2:
        out.add(("two launches", "rows" if p[0].cols == shape[1] else "columns", "split" if p[1].splits > 1 else "whole"))
    return out


def every_instance(form):
    op, kind, tB = form
    out = {(f"few_rows_n{n}", rows) for n in (16, 32, 64) for rows in (16, 32, 64) if n * rows <= 2048}
    if op == "gated" and (kind, tB) != ("e4m3", 1):  # (never the choice)
        out.remove(("few_rows_n32", 64))
    tiles = ("e4m3_pp_m256n256k128_w2x4_mt16_s2", "ep_e4m3_dma_m256n128k128_w4x2_mt16_s3",
             "ep_e4m3_dma_m128n128k128_w2x4_mt16_s4", "ep_e4m3_dma_m64n64k128_w2x2_mt16_s4") if kind == "e4m3" else \
        ("bf16_pp_m256n256k32_w2x4_mt16_s4", "bf16_dma_m256n128k64_w4x2_mt16_s3", "bf16_dma_m128n128k64_w2x4_mt16_s4",
         "bf16_dma_m64n64k64_w2x2_mt16_s4")
    for split in ("split", "whole"):
        out |= {(t, split) for t in tiles} | {("two launches", along, split) for along in ("rows", "columns")}
    return out
