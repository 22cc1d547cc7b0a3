"""Which kernel moe_linear_int8 takes for a product, as kernels_linear.hip states it; the tiles' figures
are read from there."""
import os
import re

from quantized_expert_ffn_topk_amd import abi

CUS = 256
SOURCE = os.path.join(abi.PKG, "csrc", "kernels_linear.hip")


def tiles():
    """[(tokens, channels, blocks that fit a CU, stage, fixed, alone)] of the choice."""
    text = open(SOURCE).read()
    body = re.search(r"Tile tile\[(\d+)\] = \{(.*?)\};", text, re.S)
    rows = [tuple(float(v) for v in r.split(",")) for r in re.findall(r"\{([^{}]+)\}", body.group(2))]
    assert len(rows) == int(body.group(1)) and all(len(r) == 6 for r in rows)
    return [(int(r[0]), int(r[1]), int(r[2])) + r[3:] for r in rows]


def blocks(T, N, tokens, rows):
    return -(-T // tokens) * -(-N // rows)


def tile_costs(T, N, K):
    """The choice's figure for each tile, in the tiles' order."""
    out = []
    for bt, bn, fit, stage, fixed, alone in tiles():
        n = -(-blocks(T, N, bt, bn) // CUS)
        out.append((n * stage + (alone if n % fit else 0.0)) * (K / 128.0) + -(-n // fit) * fixed)
    return out


def tile(T, N, K):
    """(tokens, channels) of the tile that is taken."""
    costs = tile_costs(T, N, K)
    return tiles()[costs.index(min(costs))][:2]


def is_stream(T, N):
    return (T <= 16 or blocks(T, N, 16, 16) <= CUS or T <= 32 or blocks(T, N, 32, 48) <= CUS
            or blocks(T, N, 64, 32) <= CUS)


def kernel(T, N, K, ldq=None, ldw=None, shift=0):
    """('stream', hint, rows, tokens, waves) or ('tiles', rows' way, hint, tokens, channels), for rows ldq and ldw
    apart that begin `shift` bytes past an address of 128 bytes' alignment."""
    ldq, ldw = ldq or K, ldw or K
    nt = N * K >= 96 << 20 and shift % 128 == 0 and ldw % 128 == 0
    if is_stream(T, N):
        tc = (1 if T <= 8 else 2 if T <= 16 or blocks(T, N, 16, 16) <= CUS
              else 4 if T <= 32 or blocks(T, N, 32, 48) <= CUS else 8)
        fits = lambda rows: blocks(T, N, 8 * tc, rows) <= CUS  # noqa: E731
        if tc == 8:
            rt, waves = 2, 8
        elif fits(16):
            rt, waves, nt = 1, 16 if tc == 1 else 8, False
        elif fits(32):
            rt, waves = 1 if tc == 1 else 2, 8
        elif fits(48):
            rt, waves = 3, 8
        elif nt and fits(64):
            rt, waves = 4, 4
        else:
            rt, waves = 3 if nt and tc > 1 else 2, 4
        return "stream", nt, 16 * rt, 8 * tc, waves
    bt, bn = tile(T, N, K)
    copies = shift % 16 == 0 and ldq % 16 == 0 and ldw % 16 == 0
    return "tiles", "copies" if copies else "registers", copies and nt and T <= bt, bt, bn
