"""Sizes at which the gated products take each form of their kernels on 152 SMs: (E, S, F, K or N).
test_gated_tile.py holds these lists to reaching every form."""

# 32-, 64- and 128-row tiles of one CTA, alone and with their reduction shared by two, four and eight; 256-row tiles of
# one CTA; 128- and 256-row tiles of a pair.  F a multiple of 16 (one copy a stage), of 8, and neither.
GATE = [(1, 5, 40, 72), (1, 5, 48, 2064), (1, 7, 35, 4112), (1, 5, 64, 16400),
        (40, 1000, 136, 72), (20, 900, 72, 2064), (8, 500, 80, 4112), (5, 250, 67, 16400),
        (40, 2500, 144, 72), (20, 1000, 136, 2064), (8, 1000, 72, 4112), (5, 250, 144, 16400),
        (40, 4000, 72, 72), (40, 6000, 136, 72), (20, 6000, 144, 72)]

BACK = [(1, 5, 40, 72), (1, 5, 48, 776), (1, 7, 35, 2064), (1, 5, 64, 16400),
        (1, 6000, 40, 72), (1, 2500, 37, 2064), (20, 900, 40, 4112), (8, 500, 48, 16400),
        (1, 16000, 40, 72), (1, 6000, 40, 2064), (1, 2500, 43, 4112), (8, 1000, 40, 16400),
        (1, 8000, 136, 72), (40, 6000, 264, 4112), (20, 16000, 136, 72)]
