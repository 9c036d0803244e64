"""Shapes (M, N, K) that reach each kernel of fp8_linear_block, with N a multiple
of four (16-byte accesses in the epilogue) and not: the CPU tests hold
linear_block_plan to this table, the GPU tests run the epilogue on it."""

KERNEL_SHAPES = {
    "rows 1x1": [(5, 1000, 272), (1, 301, 400)],
    "rows 1x2": [(7, 8000, 144), (16, 5001, 272)],
    "rows 1x4": [(9, 16400, 272), (2, 9001, 144)],
    "rows 2x1": [(60, 1000, 272), (33, 131, 400)],
    "rows 2x2": [(130, 1600, 272), (300, 516, 528), (300, 517, 144)],
    "rows 2x4": [(20, 9000, 272), (31, 9001, 144)],
    "rows 4x2": [(130, 2600, 272), (257, 1101, 144)],
    "rows 4x4": [(256, 4096, 272), (130, 5001, 144)],
    "rows 4x4 pair": [(60, 18000, 272), (50, 18001, 144)],
    "128x64": [(513, 2052, 160), (1100, 5003, 272)],
    "128x64 K2": [(505, 4004, 1408), (505, 4002, 1392)],
    "128x128": [(1500, 5004, 528), (1500, 5003, 512)],
    "128x128 K2": [(1500, 1452, 4112), (1500, 1450, 4224)],
    # more tiles than CUs, so that workgroups walk them
    "256x128": [(1020, 16380, 2064), (1020, 16379, 2048)],
}
# K = 0: no stage at all
NO_K = {"rows 2x1": [(70, 200, 0)], "rows 4x4": [(300, 3000, 0)], "128x64": [(700, 4100, 0), (2000, 5001, 0)]}
