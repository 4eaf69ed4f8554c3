"""Sizes of the gated feed-forward that reach, together with those of the
general tests, every way its products are launched: each form in each tiling,
dx and dW in one launch or two, tiles whole, cut into slices, or both in one
launch."""

BF16, F32 = 1, 0

# dtype, M, D, F
SIZES = [
    # the small tiles of the float32 forward; dx and dW by deep tiles in slices
    (F32, 10004, 8, 1056),
    # one token, weights too many for one launch: dW by big tiles
    (BF16, 1, 2144, 6992), (F32, 1, 4864, 3472), (BF16, 1, 5552, 13600),
    # one token's parts summed from big tiles
    (BF16, 37, 2512, 6704),
    # small tiles: one launch, whole and in slices
    (BF16, 9089, 528, 8), (F32, 158, 5696, 3128),
    # whole and sliced tiles of each kind in launches of their own
    (BF16, 5838, 2712, 8), (F32, 4545, 3520, 8), (F32, 1185, 6040, 168),
    (BF16, 1228, 3720, 416), (BF16, 7771, 2024, 272), (BF16, 444, 6392, 4928),
    (BF16, 13040, 1248, 1048), (F32, 3724, 144, 4552),
    # whole tiles and slices of others in one launch
    (F32, 1534, 5976, 664), (BF16, 5119, 296, 5984), (BF16, 2235, 3616, 1136),
    (BF16, 599, 2832, 10824), (BF16, 3332, 1296, 1288), (F32, 4039, 4776, 624),
    (F32, 1252, 1272, 7640), (BF16, 22157, 720, 856),
]
