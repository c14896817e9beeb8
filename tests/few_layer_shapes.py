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
