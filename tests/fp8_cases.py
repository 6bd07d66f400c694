"""Sizes that reach every kernel of the 8-bit product and gated block on 256
CUs: tokens, output channels, input channels, and the kernel's name.  Tokens
and channels end inside a tile; the blocks of k are one, odd and even numbers of
them, and more than a tile kernel loads weight scales for at a time (64, 63
with three stages, twice as many where two groups of waves share k)."""

MATMUL_16 = [
    (40, 300, 700, "few tokens"), (65, 60, 16500, "few tokens"),
    (130, 2040, 500, "64 x 64, k in two groups"), (250, 1025, 860, "64 x 64, k in two groups"),
    (70, 3001, 16500, "64 x 64, k in two groups"),
    (130, 5590, 860, "128 x 64, k in two groups"), (65, 11000, 1200, "128 x 64, k in two groups"),
    (130, 5590, 16500, "128 x 64, k in two groups"),
    (333, 5590, 100, "64 x 64"), (2043, 1025, 130, "64 x 64"), (130, 11000, 1250, "64 x 64"), (6001, 300, 8500, "64 x 64"),
    (33, 4090, 100, "128 x 128"), (517, 5590, 900, "128 x 128"), (3001, 1025, 8450, "128 x 128"),
    (333, 11000, 200, "256 x 128"), (4090, 1025, 1200, "256 x 128"), (6001, 1025, 8450, "256 x 128"),
    (700, 11000, 128, "256 x 256"), (3001, 2565, 300, "256 x 256"), (1500, 5590, 513, "256 x 256"),
    (1030, 11000, 8450, "256 x 256"),
]

MATMUL_32 = [
    (40, 300, 700, "few tokens"), (65, 60, 16500, "few tokens"),
    (65, 5590, 500, "64 x 64, k in two groups"), (33, 8190, 860, "64 x 64, k in two groups"),
    (130, 3001, 16500, "64 x 64, k in two groups"),
    (6001, 130, 300, "128 x 64, k in two groups"), (65, 11000, 860, "128 x 64, k in two groups"),
    (130, 5590, 16500, "128 x 64, k in two groups"),
    (49001, 64, 100, "64 x 64"), (130, 11000, 1250, "64 x 64"), (6001, 300, 8500, "64 x 64"),
    (33, 4090, 100, "256 x 128"), (517, 5590, 300, "256 x 128"), (333, 11000, 1200, "256 x 128"),
    (6001, 1025, 8450, "256 x 128"),
    (700, 11000, 128, "256 x 256"), (3001, 2565, 300, "256 x 256"), (1500, 5590, 2600, "256 x 256"),
    (4090, 2565, 8450, "256 x 256"),
]

_IN_TWO = ", then the quantizer"
GATED = [
    (5, 300, 700, "few tokens" + _IN_TWO), (65, 60, 900, "few tokens" + _IN_TWO),
    (65, 2040, 600, "32 channels x 64, k in two groups" + _IN_TWO),
    (33, 5590, 860, "32 channels x 64, k in two groups" + _IN_TWO),
    (130, 2040, 16500, "32 channels x 64, k in two groups" + _IN_TWO),
    (70, 5590, 860, "64 channels x 64, k in two groups" + _IN_TWO),
    (333, 1500, 1250, "64 channels x 64, k in two groups" + _IN_TWO),
    (70, 5590, 16500, "64 channels x 64, k in two groups" + _IN_TWO),
    (65, 516, 200, "128 channels x 64"), (130, 5590, 1250, "128 channels x 64"), (65, 11000, 8450, "128 channels x 64"),
    (333, 5590, 300, "128 channels x 128"), (130, 11000, 1250, "128 channels x 128"), (6001, 300, 8450, "128 channels x 128"),
    (333, 11000, 300, "128 channels x 256"), (12001, 300, 1250, "128 channels x 256"),
    (6001, 1025, 8450, "128 channels x 256"),
]


def matmul(types=("float16", "bfloat16", "float32")):
    """(tokens, output channels, input channels, kernel, output type)"""
    return [case + (t,) for t in types for case in (MATMUL_32 if t == "float32" else MATMUL_16)]


def batches(cases):
    """The cases that keep their kernel when the first token is left out."""
    return [c for c in cases if c[0] % 32 != 1]
