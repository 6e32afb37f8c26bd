"""Sizes for which the plans of the operators on 8-bit codes choose every kernel
instance that they can choose, with ends inside tiles and steps.

FORWARD and BACKWARD: rows, Cin, Cout; ROWS: columns. The instances that they
have to reach: tiles, + k split; "rows" the kernel of one or two rows,
thin16 and thin32 those of short batches; lanes x
steps of a row held in registers, 0x0 one that is read twice."""

FORWARD = [(1, 145, 37), (2, 145, 37), (4, 1451, 97), (5, 175, 37), (5, 1551, 41), (5, 4091, 1109), (8512, 143, 71), (4134, 2811, 35),
           (514, 139, 6649), (154, 6569, 5551), (8257, 519, 1555), (1864, 7473, 2179),
           (16, 4091, 333), (38, 139, 8209), (3, 12835, 41), (97, 9697, 2659), (144, 7326, 6005)]
FORWARD_INSTANCES = {"rows", "thin16", "thin32", "64x64", "64x64+", "128x64", "128x64+", "128x128", "128x128+", "256x256", "256x256+"}

BACKWARD = {
    "f32": [(33, 139, 43), (917, 177, 37), (35, 189, 925), (33, 3627, 491), (6172, 267, 35), (33, 367, 4943), (553, 323, 4925),
            (7484, 195, 627), (2281, 4535, 2489)],
    "bf16": [(33, 187, 39), (1745, 185, 37), (34, 157, 1717), (36, 7515, 219), (7953, 227, 35), (33, 549, 3351), (1401, 213, 7791),
             (7057, 221, 1837), (2738, 6759, 3041)],
}
BACKWARD_INSTANCES = {f"{o}={t}" for o in ("dw", "dx") for t in ("64x64", "64x64+", "128x64", "128x64+", "128x128", "128x128+", "256x128")}

ROWS = [7, 512, 600, 1200, 2000, 2100, 2600, 3100, 5000, 7000, 9000, 15000, 30000, 40000]
ROWS_INSTANCES = {f"f={s}" for s in ("64x1", "64x2", "64x3", "64x4", "64x5", "64x6", "64x8", "256x3", "256x4", "256x5", "256x8", "1024x4",
                                     "0x0")} | {f"b={s}" for s in ("64x1", "64x2", "64x3", "64x4", "256x2", "512x2", "1024x2", "0x0")}
