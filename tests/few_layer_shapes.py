"""Sizes of the few-token layer's tests with the kernels that they are there
for (checked on the CPU by test_few_plan.py, run by test_gpu_few_forms.py)."""

# (tokens, experts, k): the experts are picked inside the first product.  Odd
# numbers of experts, each count of threads per expert, several tokens one
# after the other; the largest on each edge of the rule, and the smallest
# past it
PICKS = {(1, 5, 3): True, (2, 5, 5): True, (3, 33, 4): True,
         (4, 5, 2): True, (4, 32, 32): True, (3, 61, 8): True,
         (4, 64, 8): True, (4, 128, 8): True, (3, 170, 6): True,
         (2, 255, 20): True, (2, 256, 8): True, (1, 256, 32): True,
         (4, 129, 8): False, (3, 171, 6): False, (3, 256, 4): False,
         (1, 257, 8): False, (2, 300, 5): False, (1, 512, 32): False,
         (4, 1024, 8): False, (2, 1024, 32): False, (5, 5, 2): False}

# (tokens, H, F, experts, k, format, scales at dwords) -> dword scales, tokens
# of a column set, column sets, a wave per item
FORMS = {
    # MXFP4 with dword scales: waves sharing an item
    (1, 384, 128, 8, 2, "mxfp4", True): (True, 2, 1, False),
    (2, 128, 1408, 8, 4, "mxfp4", True): (True, 2, 1, False),
    (6, 128, 256, 40, 3, "mxfp4", True): (True, 2, 1, False),
    (16, 640, 256, 64, 4, "mxfp4", True): (True, 2, 2, False),
    (13, 128, 384, 7, 2, "mxfp4", True): (True, 8, 1, False),
    (32, 384, 128, 8, 1, "mxfp4", True): (True, 8, 1, False),
    (40, 256, 128, 5, 2, "mxfp4", True): (True, 8, 2, False),
    (64, 128, 640, 4, 3, "mxfp4", True): (True, 8, 2, False),
    # a wave per item: few and many chunks, FFN columns that end inside one
    (8, 128, 8320, 16, 1, "mxfp4", True): (True, 2, 1, True),
    (2, 128, 32768, 2, 1, "mxfp4", True): (True, 2, 1, True),
    (16, 128, 768, 128, 8, "mxfp4", True): (True, 2, 2, True),
    (12, 384, 1408, 48, 4, "mxfp4", True): (True, 2, 2, True),
    (32, 128, 768, 128, 8, "mxfp4", True): (True, 8, 1, True),
    (8, 384, 8832, 8, 2, "mxfp4", True): (True, 8, 1, True),
    (33, 128, 8192, 8, 2, "mxfp4", True): (True, 8, 2, True),
    (64, 384, 16384, 4, 2, "mxfp4", True): (True, 8, 2, True),
    # byte scales: sizes that are no multiples of 128, scales between dwords
    (1, 96, 160, 6, 2, "mxfp4", True): (False, 2, 1, False),
    (2, 128, 256, 6, 2, "mxfp4", False): (False, 2, 1, False),
    (19, 128, 256, 6, 2, "mxfp4", False): (False, 8, 1, False),
    (2, 64, 32800, 3, 2, "mxfp4", True): (False, 2, 1, True),
    (9, 96, 4128, 24, 4, "mxfp4", True): (False, 8, 1, True),
    (17, 128, 768, 128, 6, "mxfp4", False): (False, 8, 1, True),
    # bf16
    (3, 72, 40, 6, 2, "bf16", True): (False, 8, 1, False),
    (8, 128, 8200, 8, 2, "bf16", True): (False, 8, 1, False),
    (24, 136, 264, 6, 1, "bf16", True): (False, 8, 1, False),
    (24, 136, 264, 6, 2, "bf16", True): (False, 8, 2, False),
    (40, 264, 72, 4, 2, "bf16", True): (False, 8, 4, False),
    (64, 128, 1000, 8, 2, "bf16", True): (False, 8, 4, False),
    (24, 64, 4360, 8, 2, "bf16", True): (False, 8, 2, True),
    (64, 136, 4104, 16, 2, "bf16", True): (False, 8, 2, True),
    (33, 72, 8200, 4, 2, "bf16", True): (False, 8, 4, True),
    (64, 520, 4104, 8, 3, "bf16", True): (False, 8, 4, True)}
