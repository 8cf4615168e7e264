"""Sizes at which the output head's losses take each of their forms, shared by the tests that run them and by the one
that holds them to those forms.

A call's form follows from its sizes: logits in tiles of 64, 128 or 256 columns, on the caller's x (up to 128 tokens) or
on a copy of its rows with a target; the backward in pieces of the vocabulary.
"""
# name: tokens, vocabulary, hidden, columns of a tile of logits, whether the backward takes the caller's x
FORMS = {
    "10 on x": (10, 3001, 328, 64, True),
    "30 on x": (30, 2999, 328, 64, True),
    "50 on x": (50, 3070, 328, 64, True),
    "65 on x": (65, 33001, 1000, 128, True),
    "100 on x": (100, 14501, 2312, 64, True),
    "128 on x": (128, 66003, 504, 128, True),
    "100 copied": (100, 4001, 328, 64, False),
    "300 in 128": (300, 9001, 264, 128, False),
    "300 in 256": (300, 24577, 264, 256, False),  # (dx in 128)
    "700 in 256": (700, 16701, 1000, 256, False),
}
# w larger than the last-level cache, 256 MiB
STREAMED = {"40 streamed": (40, 140001, 1000, 64, True), "100 streamed": (100, 140001, 1000, 128, True)}
# tokens, vocabulary, hidden, columns of a piece of f32 gradients
PIECES = (4000, 24577, 264, 12544)
# tokens, vocabulary: the same rows in a part of the batch take narrower tiles
BATCH = (1000, 12500, {1: 64, 64: 64, 100: 64, 200: 128, 1000: 256})

THREE_PARTS = 1.7e-6  # bound of the relative error of f32 gradients, by the norm (test_three_parts)
