"""Sizes of grouped products that reach each kernel.  tests/test_plan_cpu.py holds
them to the rules that choose, and the GPU tests run them."""

# name: (kernel, rows of each expert, rows before the groups and behind them, N, K, group size).
# The streaming kernels' sizes give a workgroup several blocks of weight rows (256 of them share the
# pieces' N / 16 blocks), and pieces that change among them; the tiles' groups end in each quarter of a tile.
EXPERTS = {
    "stream1": ("stream1", [9, 0, 20, 1, 3, 8], 2, 3, 8200, 96, 32),
    "stream1-long": ("stream1", [0, 1, 17, 40, 2, 3, 0, 5, 1, 6, 4, 1], 1, 2, 2057, 2080, 32),
    "stream1-most": ("stream1", [33, 0, 3, 1, 0, 2, 2, 1], 1, 0, 1037, 4096, 128),
    "stream2": ("stream2", [35, 0, 17, 2, 1, 3], 2, 2, 8200, 512, 64),
    "stream2-odd": ("stream2", [33, 16, 0, 5, 0, 1], 0, 1, 8213, 1184, 32),
    "stream2-long": ("stream2", [40, 0, 17, 3, 1, 2, 16, 5], 1, 3, 4105, 2080, 32),
    "stream2-most": ("stream2", [33, 0, 8, 1], 1, 2, 2056, 4096, 128),
    "skinny": ("skinny", [9, 0, 17, 2, 1, 33], 2, 1, 136, 4224, 128),
    "skinny-odd": ("skinny", [1, 0, 31, 5], 1, 3, 57, 4128, 32),
    "skinny-one": ("skinny", [1], 0, 0, 15, 8256, 64),
    "tile64": ("tile64", [100, 0, 1, 64, 65, 17], 3, 70, 200, 352, 32),
    "tile128": ("tile128", [300, 0, 1, 129, 128, 60, 70, 350], 3, 40, 2056, 96, 32),
    "tile128-odd": ("tile128", [140, 97, 0, 485, 33, 96], 1, 70, 2059, 320, 64),
    "tile256": ("tile256", [900, 0, 1, 256, 200, 150, 70, 2500], 3, 130, 2056, 96, 32),
    "tile256-odd": ("tile256", [1400, 129, 0, 64, 193, 2400], 1, 260, 2059, 320, 64),
}

# The same for the gradients: (rows of a whole piece, rows of each expert, before, behind, N, K, group size).
EXPERTS_DX = {
    "short": (64, [100, 0, 1, 64, 65, 17], 3, 70, 200, 352, 32),
    "short-few": (64, [1, 0, 3, 2], 1, 2, 1032, 96, 32),
    "whole": (256, [300, 0, 70, 150, 200, 1, 256, 330], 3, 130, 72, 1664, 128),
    "whole-odd": (256, [65, 129, 193, 257, 0, 440], 1, 260, 264, 2208, 32),
}

# name: (the product's kernel, M, N, K, group size)
LORA = {
    "skinny": ("skinny", 5, 4200, 96, 32),
    "skinny-blocks3": ("skinny", 16, 8200, 320, 64),
    "skinny-blocks4": ("skinny", 9, 12403, 96, 32),
    "skinny-two": ("skinny", 30, 8201, 96, 32),
    "skinny-two-blocks4": ("skinny", 32, 12400, 96, 32),
    "skinny-four": ("skinny", 60, 4203, 320, 64),
    "skinny-slices": ("skinny", 95, 8200, 96, 32),
    "skinny-slices-blocks4": ("skinny", 96, 12403, 96, 32),
    "tile64": ("tile64", 300, 520, 96, 32),
    "tile64-parts": ("tile64", 130, 259, 1184, 32),
    "tile128": ("tile128", 300, 8200, 96, 32),
    "tile128-odd": ("tile128", 97, 16403, 96, 32),
    "tile128-more": ("tile128", 600, 5603, 320, 64),
    "tile256": ("tile256", 1030, 6664, 96, 32),
    "tile256-odd": ("tile256", 2100, 4107, 320, 64),
}

# name: (rows of a tile of the gradient, parts of N, M, N, K, group size)
LORA_DX = {
    "rows64": (64, 1, 300, 136, 352, 32),
    "rows64-parts": (64, 4, 300, 2056, 384, 128),
    "rows128": (128, 1, 600, 136, 3200, 64),
    "rows256": (256, 1, 1300, 72, 3232, 32),
    "rows256-long": (256, 1, 1100, 1096, 3328, 128),
}
