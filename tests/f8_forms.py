"""Which kernel f8_linear takes, by the rule of decode/f8.hip on 256 compute units, and sizes that reach each of them."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "dense_fp16_gemm_hgemm_amd", "decode", "f8.hip")
CUS = 256


def tiles():
    """(rows, columns, us) of the tiles for many tokens, as the source has them."""
    text = open(SOURCE, encoding="utf-8").read()
    found = re.search(r"kTiles\[\] = \{(.*?)\};", text, flags=re.S).group(1)
    return [(int(m), int(n), float(us)) for m, n, us in re.findall(r"\{(\d+), (\d+), ([\d.]+)f\}", found)]


def up(a, b):
    return -(-a // b)


def form(M, N, K, multiple=None):
    """The kernel's name.  multiple: of how many bytes rows begin and end at multiples (contiguous rows: of K's power of two)."""
    multiple = K & -K if multiple is None else multiple
    if K < 16:
        return "short"
    narrow = up(N, 16) <= CUS
    if multiple % 4:
        if M <= 16 and narrow:
            return "any"
        return "loose 64x64" if up(M, 64) * up(N, 64) <= 3 * CUS else "loose 128x128"
    for most, wide in ((16, "1x2 of 12"), (32, "2x4 of 4"), (64, "4x4 of 4")):
        if M <= most:
            return "strip " + ({16: "1x1 of 16", 32: "2x1 of 12", 64: "4x1 of 6"}[most] if narrow else wide)
    best, least = 0, float("inf")
    for i, (bm, bn, us) in enumerate(tiles()):
        t = up(up(M, bm) * up(N, bn), CUS) * us
        if t <= least and (i < 5 or multiple % 16 == 0) and (i > 0 or M <= 64 * 65535):
            best, least = i, t
    bm, bn, _ = tiles()[best]
    return ("strip 4x2 of 6", f"tile {bm}x{bn}", f"turns {bm}x{bn}")[0 if best == 0 else 2 if best == 5 else 1]


def waves(name):
    """Waves that share K in a strip."""
    return int(name.split()[-1])


FORMS = {"short", "any", "loose 64x64", "loose 128x128", "strip 1x1 of 16", "strip 1x2 of 12", "strip 2x1 of 12", "strip 2x4 of 4",
         "strip 4x1 of 6", "strip 4x4 of 4", "strip 4x2 of 6", "tile 64x64", "tile 64x128", "tile 128x128", "tile 128x256", "turns 256x256"}

# One block of 128 columns, part of one, numbers that fill a ring or not, odd and even ones; last tiles in part.
SIZES = [
    (512, 4096, 1024), (500, 4090, 1168), (128, 14336, 272), (100, 14300, 16), (510, 4000, 144),    # 64 x 128
    (4096, 4096, 16), (4096, 4096, 128), (4096, 4096, 256), (4000, 4090, 1040), (3900, 4096, 1168),  # 256 x 256
    (4096, 8192, 400),
    (4096, 4096, 20), (3990, 4050, 1036),                                                           # rows at multiples of 4
    (1024, 4096, 16), (1024, 4096, 256), (1000, 4096, 272), (1020, 4000, 1040), (1024, 4090, 520),                     # 128 x 128
    (2048, 4096, 16), (2000, 4080, 400), (2047, 4096, 648), (512, 14336, 272),                      # 128 x 256
    (256, 4096, 16), (200, 4096, 128), (256, 4000, 656), (250, 4096, 780),                          # 64 x 64
    (128, 4096, 16), (100, 4000, 144), (128, 4096, 912), (70, 8000, 1300),                          # 64 x 32
]
# A wave that is alone with K takes more than 64 of its blocks: the weights' scales are read anew.
LONG = [(3, 70, 131500), (5, 5000, 98600), (20, 100, 98700), (25, 8000, 33300), (50, 300, 50000), (60, 6000, 33000), (100, 300, 49700)]
# Rows at odd bytes: more than 32 blocks, which are two trips of a workgroup's sixteen waves.
ODD = [(1, 300, 8191), (16, 4096, 4225), (7, 40, 12801), (100, 300, 4097), (1100, 4100, 1031), (900, 5000, 21)]
