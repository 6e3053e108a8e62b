"""The forms of the block-scaled FP8 products, with a product for each.

A form is
    ("streaming", tokens of a tile, CTAs of a row block, CTAs an SM, more groups than ring stages)
    ("pairs" or "single", CTAs of a tile, more tiles than are in flight)
and the products are small, with part tiles of tokens and rows and a shorter last group.
"""
import ctypes

import swiglu_mlp_dfk_b200 as dfk

SMS = 148

PLAIN = [  # (M, K, N)
    ((5, 272, 130), ("streaming", 16, 1, 2, False)),
    ((5, 784, 130), ("streaming", 16, 1, 2, True)),
    ((5, 1040, 130), ("streaming", 16, 2, 2, False)),
    ((5, 2064, 12297), ("streaming", 16, 2, 2, True)),
    ((5, 2064, 130), ("streaming", 16, 4, 2, False)),
    ((5, 3088, 130), ("streaming", 16, 4, 2, True)),
    ((5, 4112, 130), ("streaming", 16, 8, 2, False)),
    ((5, 6160, 130), ("streaming", 16, 8, 2, True)),
    ((24, 272, 130), ("streaming", 32, 1, 2, False)),
    ((24, 656, 130), ("streaming", 32, 1, 2, True)),
    ((24, 1040, 130), ("streaming", 32, 2, 2, False)),
    ((24, 2064, 12297), ("streaming", 32, 2, 2, True)),
    ((24, 2064, 130), ("streaming", 32, 4, 2, False)),
    ((24, 3088, 130), ("streaming", 32, 4, 2, True)),
    ((24, 4112, 130), ("streaming", 32, 8, 2, False)),
    ((24, 6160, 130), ("streaming", 32, 8, 2, True)),
    ((50, 272, 130), ("streaming", 64, 1, 2, False)),
    ((50, 528, 130), ("streaming", 64, 1, 2, True)),
    ((50, 1008, 130), ("streaming", 64, 2, 2, False)),
    ((50, 1040, 130), ("streaming", 64, 2, 2, True)),
    ((50, 2032, 130), ("streaming", 64, 4, 2, False)),
    ((50, 2064, 130), ("streaming", 64, 4, 2, True)),
    ((50, 4080, 130), ("streaming", 64, 8, 2, False)),
    ((50, 4112, 130), ("streaming", 64, 8, 2, True)),
    ((70, 272, 19217), ("single", 1, False)),
    ((70, 272, 38417), ("single", 1, True)),
    ((1100, 4112, 1089), ("single", 2, False)),
    ((520, 6160, 1089), ("single", 4, False)),
    ((330, 272, 6465), ("pairs", 2, False)),
    ((150, 272, 19217), ("pairs", 2, True)),
    ((13, 14352, 1001), ("streaming", 16, 8, 2, True)),
]
GATED = [  # (M, d_model, d_ff)
    ((5, 272, 400), ("streaming", 16, 1, 1, False)),
    ((5, 784, 400), ("streaming", 16, 1, 1, True)),
    ((5, 272, 19216), ("streaming", 16, 1, 2, False)),
    ((5, 400, 19216), ("streaming", 16, 1, 2, True)),
    ((5, 1040, 400), ("streaming", 16, 2, 1, False)),
    ((5, 2064, 5008), ("streaming", 16, 2, 1, True)),
    ((5, 2064, 400), ("streaming", 16, 4, 1, False)),
    ((5, 3088, 400), ("streaming", 16, 4, 1, True)),
    ((5, 4112, 400), ("streaming", 16, 8, 1, False)),
    ((5, 6160, 400), ("streaming", 16, 8, 1, True)),
    ((24, 272, 400), ("streaming", 32, 1, 1, False)),
    ((24, 784, 400), ("streaming", 32, 1, 1, True)),
    ((24, 272, 19216), ("streaming", 32, 1, 2, False)),
    ((24, 400, 19216), ("streaming", 32, 1, 2, True)),
    ((24, 1040, 400), ("streaming", 32, 2, 1, False)),
    ((24, 2064, 5008), ("streaming", 32, 2, 1, True)),
    ((24, 2064, 400), ("streaming", 32, 4, 1, False)),
    ((24, 3088, 400), ("streaming", 32, 4, 1, True)),
    ((24, 8208, 400), ("streaming", 32, 8, 1, True)),
    ((50, 272, 400), ("streaming", 64, 1, 1, False)),
    ((50, 656, 400), ("streaming", 64, 1, 1, True)),
    ((50, 1040, 400), ("streaming", 64, 2, 1, False)),
    ((520, 2064, 656), ("streaming", 64, 2, 1, True)),
    ((50, 2064, 400), ("streaming", 64, 4, 1, False)),
    ((50, 3088, 400), ("streaming", 64, 4, 1, True)),
    ((50, 8208, 400), ("streaming", 64, 8, 1, True)),
    ((520, 272, 3088), ("single", 1, False)),
    ((70, 272, 19216), ("single", 1, True)),
    ((520, 4112, 1040), ("single", 2, False)),
    ((520, 6160, 656), ("single", 4, False)),
    ((1100, 272, 1040), ("pairs", 2, False)),
    ((1100, 272, 2064), ("pairs", 2, True)),
    ((5, 4112, 14352), ("streaming", 16, 1, 1, True)),
    ((24, 4112, 14352), ("streaming", 32, 1, 1, True)),
    ((300, 4112, 1040), ("streaming", 64, 2, 1, True)),
]


def form(nmat, M, K, N, sms=SMS):
    """The form that a product of nmat weight matrices takes."""
    out = (ctypes.c_int * 5)()
    dfk.lib().dfk_fp8_block_form(nmat, M, K, N, sms, out)
    groups = -(-K // 128)
    if out[0]:
        return ("streaming", out[1], out[2], 1 + out[3], -(-groups // out[2]) > out[4])
    tiles = -(-M // (256 if out[1] else 128)) * -(-N // (128 if nmat == 2 else 256))
    # where CTAs share a tile, every tile is in flight
    return ("pairs" if out[1] else "single", out[2],
            tiles > (sms // 2 if out[1] else sms) and (out[1] == 1 or out[2] == 1))
