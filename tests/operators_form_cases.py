"""Calls that between them take every form of the operators around the scan: the kernels' variants that
the plans choose from the sizes (test-only)."""

# M, N, K, out, the form: ("few", 16-row groups of a per wave, waves), or ("big", 16-row groups of a per wave,
# whether the sum over k is split). Each with b's scales in either layout.
MATMUL = [
    (5, 9001, 300, "bf16", ("few", 1, 4)), (5, 9001, 300, "f32", ("few", 1, 4)),
    (3, 1503, 2200, "bf16", ("few", 1, 16)), (16, 700, 4900, "f32", ("few", 1, 16)),
    (20, 9001, 1300, "bf16", ("few", 2, 4)), (20, 9001, 1300, "f32", ("few", 2, 4)),
    (31, 3001, 2200, "bf16", ("few", 2, 8)), (18, 1500, 1160, "f32", ("few", 2, 8)),
    (64, 9001, 1300, "bf16", ("few", 4, 4)), (33, 9001, 1300, "f32", ("few", 4, 4)),
    (40, 600, 2200, "bf16", ("few", 4, 8)), (64, 700, 1300, "f32", ("few", 4, 8)),
    (300, 300, 400, "bf16", ("big", 4, False)), (300, 300, 400, "f32", ("big", 4, False)),
    (999, 1000, 16399, "bf16", ("big", 4, True)), (260, 260, 20000, "f32", ("big", 4, True)),
    (4001, 3999, 1000, "bf16", ("big", 8, False)), (3000, 4001, 4096, "bf16", ("big", 8, False)),
    (1290, 1289, 33000, "bf16", ("big", 8, True)), (2050, 2051, 16384, "bf16", ("big", 8, True)),
]
MATMUL_FORMS = {("few", mb, waves, out) for mb in (1, 2, 4) for waves in (4, 16 if mb == 1 else 8) for out in ("bf16", "f32")}
MATMUL_FORMS |= {("big", mb, split, out) for mb in (4, 8) for split in (False, True) for out in ("bf16", "f32")
                 if mb == 4 or out == "bf16"}

# B, T, C, kind, the forms forwards and backwards: (channels per lane, segmented, walked by lanes)
GATED = [
    (9, 300, 70, "f32", (1, False, False), (1, False, False)),
    (2, 1300, 70, "f32", (1, True, False), (1, True, False)),
    (9, 300, 71, "bf16", (1, False, False), (1, False, False)),
    (3, 1100, 71, "bf16", (1, True, False), (1, True, False)),
    (9, 300, 258, "bf16", (2, False, False), (2, False, False)),
    (3, 1100, 258, "bf16", (2, True, False), (2, True, False)),
    (5, 7, 70, "f32", (1, False, True), (1, False, False)),
    (5, 7, 71, "bf16", (1, False, True), (1, False, False)),
    (300, 31, 70, "f32", (1, False, True), (1, False, False)),
    (300, 31, 70, "bf16", (1, False, True), (2, False, False)),
]
GATED_FORMS = {(1, seg, False, kind) for seg in (False, True) for kind in ("f32", "bf16")}
GATED_FORMS |= {(2, seg, False, "bf16") for seg in (False, True)}
GATED_WALKS = {(1, False, True, kind) for kind in ("f32", "bf16")}

# rows, F, kind: for every number of lanes per row, more rows than the workgroups hold at once (forwards at most
# 2048 workgroups of 16, 4 or 1 rows, backwards fewer)
NORM = [(33001, 100, "bf16"), (33001, 61, "f32"), (8300, 500, "bf16"), (8300, 333, "f32"), (8300, 1000, "bf16"),
        (8300, 520, "f32"), (2500, 2000, "bf16"), (2500, 1030, "f32"), (2500, 4096, "bf16"), (2500, 2100, "f32"),
        (2500, 5000, "bf16"), (2500, 8192, "f32"), (2300, 9000, "bf16"), (2300, 16384, "f32")]
