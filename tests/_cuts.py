"""Sizes at which the attention tiles' keys are cut unevenly: `cut` = (pieces,
64ths in each but the last).  L: the keys that the call is laid out for."""

CASES = {
    "86 heads of 64, 1600 keys": dict(B=1, Lq=70, Hq=86, H=86, D=64, L=1600, cut=(3, 30)),
    "2 x 75 shared heads of 64, 1984 keys": dict(B=2, Lq=33, Hq=150, H=75, D=64, L=1984, cut=(2, 48)),
    "75 heads of 64, 7936 keys": dict(B=1, Lq=64, Hq=75, H=75, D=64, L=7936, cut=(4, 20)),
    "130 heads of 128, 1280 keys": dict(B=1, Lq=65, Hq=130, H=130, D=128, L=1280, cut=(2, 48)),
}


def row_tiles(c):
    return c["B"] * c["H"] * -(-c["Lq"] * (c["Hq"] // c["H"]) // 256)
