"""Sizes that take every kernel of the tiled 8-bit linear products, and what
the planner has to choose for them: shared by the GPU test that runs them and
the CPU test that asks the planner."""

Y, DW, DX = 0, 1, 2

# pass, tokens, out, in, dy is fp32, dy's rows are whole 16-byte pieces,
# (tile, form of the 8-bit operand, share of the tiles that is split)
CASES = [
    (Y, 207, 211, 523, False, True, (128, "converted", "none")),
    (Y, 405, 419, 3633, False, True, (128, "converted", "all")),
    (Y, 4151, 1986, 3040, False, True, (128, "converted", "some")),
    (Y, 8244, 925, 551, False, True, (256, "converted", "none")),
    (Y, 900, 4200, 6800, False, True, (256, "converted", "all")),
    (Y, 4300, 4340, 20001, False, True, (256, "converted", "some")),
    (DW, 262, 200, 258, False, True, (128, "converted", "none")),
    (DW, 8347, 264, 215, False, True, (128, "converted", "all")),
    (DW, 2948, 1114, 7606, False, False, (128, "converted", "some")),
    (DW, 257, 3140, 268, True, True, (128, "cut", "none")),
    (DW, 8332, 195, 212, True, False, (128, "cut", "all")),
    (DW, 303, 7488, 1054, False, True, (256, "converted", "none")),
    (DW, 8192, 2304, 768, False, True, (256, "converted", "all")),
    (DW, 5655, 427, 3296, False, False, (256, "converted", "all")),
    (DW, 1357, 399, 5614, True, False, (256, "converted", "all")),
    (DW, 651, 7904, 1117, False, True, (256, "expanded", "none")),
    (DW, 2191, 5605, 652, False, False, (256, "expanded", "all")),
    (DW, 1171, 7080, 2421, False, True, (256, "expanded", "some")),
    (DW, 689, 3729, 5872, True, False, (256, "expanded", "some")),
    (DX, 215, 263, 207, False, False, (128, "converted", "none")),
    (DX, 222, 8555, 195, False, False, (128, "converted", "all")),
    (DX, 924, 2791, 8471, False, False, (128, "converted", "some")),
    (DX, 4553, 266, 260, True, False, (128, "cut", "none")),
    (DX, 222, 8555, 195, True, False, (128, "cut", "all")),
    (DX, 1287, 264, 6177, False, True, (256, "converted", "none")),
    (DX, 402, 2200, 8730, False, True, (256, "converted", "all")),
    (DX, 683, 782, 5473, True, False, (256, "converted", "all")),
    (DX, 7500, 664, 1086, False, True, (256, "expanded", "none")),
    (DX, 5651, 3696, 398, False, True, (256, "expanded", "all")),
    (DX, 2386, 1037, 7109, False, False, (256, "expanded", "some")),
    (DX, 5852, 697, 3620, True, False, (256, "expanded", "some")),
]


def planes(case):
    """What the planner is told of dy: 0 it is used as it lies, 1 its rows are
    laid out first, 3 it is cut into three pieces."""
    _pass, _t, n, _k, f32, whole, _ = case
    return 0 if case[0] == Y else 3 if f32 else 0 if whole and n % 8 == 0 else 1
