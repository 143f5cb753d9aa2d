"""Sizes (M, N, K) of svdq_gemm_act_residual by the kernel they reach, in every type: its tiles, whether
K is split, and how the last partial round of 256 x 256 tiles is cut.  Ragged: M and N end inside
tiles, K inside a stage of 128 bytes."""
CASES = [
    ("few rows", False, 0, (5, 121, 528)), ("few rows", False, 0, (25, 162, 656)), ("few rows", False, 0, (42, 505, 304)),
    ("few rows", False, 0, (61, 204, 816)),
    ("64x64", False, 0, (293, 499, 176)), ("64x64", False, 0, (890, 258, 112)),
    ("64x64", True, 0, (68, 56, 4016)), ("64x64", True, 0, (481, 102, 6608)),
    ("64x128", False, 0, (1997, 4703, 304)), ("64x128", False, 0, (154, 9131, 2032)),
    ("64x128", True, 0, (69, 2709, 8064)), ("64x128", True, 0, (130, 2966, 10256)), ("64x128", True, 0, (350, 1253, 9024)),
    ("128x192", False, 0, (1410, 7468, 880)), ("128x192", False, 0, (1907, 3052, 1584)),
    ("128x256", False, 0, (1394, 5045, 336)), ("128x256", False, 0, (2979, 2365, 336)),
    ("256x256", False, 0, (1931, 8134, 80)), ("256x256", False, 0, (4030, 3931, 160)),
    ("256x256", False, 1, (2665, 4793, 976)),               # a partial round alone
    ("256x256", False, 1, (3918, 7107, 272)),               # behind a whole one, as below
    ("256x256", False, 2, (3374, 6804, 304)), ("256x256", False, 2, (4204, 5501, 304)),
    ("256x256", False, 4, (4185, 4550, 160)), ("256x256", False, 4, (2731, 6857, 176)),
]
TYPE_CODES = {"int8": 3, "e4m3": 4, "f16": 0, "bf16": 1}
