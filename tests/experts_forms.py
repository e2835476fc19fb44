"""Sizes at which the experts' products take each form of their kernels on 152 SMs: (load, E, S, N, K), loads as
counts_case() of test_gpu_experts.py names them.  test_experts_tile.py holds these lists to reaching every form."""

# 32-, 64- and 128-row tiles of one CTA, alone and with their reduction shared by two, four and eight; 256-row tiles of
# one CTA; 128- and 256-row tiles of a pair
PRODUCTS = [("spread", 1, 7, 72, 200), ("spread", 1, 5, 72, 2064), ("spread", 1, 30, 80, 4112), ("spread", 1, 9, 72, 16400),
            ("gaps", 40, 1000, 264, 200), ("spread", 20, 1000, 136, 2064), ("gaps", 8, 500, 136, 4112),
            ("spread", 5, 250, 136, 16400),
            ("gaps", 40, 2500, 264, 200), ("spread", 20, 1000, 264, 2064), ("gaps", 8, 1000, 136, 4112),
            ("spread", 5, 250, 264, 16400),
            ("spread", 40, 4000, 136, 200), ("gaps", 40, 4000, 264, 200), ("spread", 40, 8000, 136, 200)]

# 128- and 256-row tiles of one CTA and of a pair (rows: N, columns: K)
GRADIENTS = [("spread", 3, 200, 72, 72), ("gaps", 4, 300, 40, 136), ("spread", 5, 20, 2000, 264), ("gaps", 5, 620, 2000, 264),
             ("spread", 5, 20, 136, 2000), ("spread", 3, 900, 264, 1000)]

# 8-bit products through widened copies: the tiles that a batch of more than 128 rows an expert takes
COPIED = [("spread", 1, 150, 72, 200), ("spread", 1, 150, 72, 2064), ("spread", 1, 150, 72, 4112), ("spread", 1, 2500, 136, 200),
          ("spread", 1, 2500, 72, 2064), ("spread", 1, 700, 136, 4112), ("spread", 1, 16000, 72, 200),
          ("spread", 1, 2500, 136, 2064), ("spread", 1, 2500, 72, 4112), ("spread", 1, 4000, 264, 200), ("gaps", 5, 1000, 2000, 200),
          ("gaps", 5, 1000, 2000, 4112), ("spread", 1, 500, 4090, 4096)]

# 8-bit products widened on the way (17 to 128 rows an expert): tiles of 32, 64 and 128 rows, one to eight CTAs a reduction
WIDENED = [("spread", 1, 20, 72, 200), ("spread", 1, 20, 72, 520), ("spread", 1, 17, 80, 1040), ("spread", 1, 25, 72, 4112),
           ("gaps", 40, 1000, 264, 200), ("spread", 20, 1000, 136, 520), ("gaps", 8, 500, 136, 1040), ("spread", 5, 250, 136, 4112),
           ("spread", 40, 4000, 136, 200), ("gaps", 20, 2500, 136, 520), ("spread", 20, 2500, 72, 1040), ("gaps", 8, 500, 136, 4112)]
