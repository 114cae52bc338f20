"""Shapes of the shared-prefix call, one for each way it can be cut: (form, d, most rows of the
kernel's form) -> (B, steps, q_heads, kv_heads, d, prefix, capacity), and the plan that the
library has to give for it, (parts, workers, in_list)."""
import random

FORMS = {
    # the prefix as one more sequence of the cache pass
    ("list", 64, 8): ((1, 2, 4, 2, 64, 165, 109), (0, 148, True)),
    ("list", 64, 16): ((2, 3, 4, 2, 64, 165, 169), (0, 148, True)),
    ("list", 64, 32): ((2, 3, 12, 3, 64, 109, 166), (0, 148, True)),
    ("list", 128, 8): ((2, 1, 6, 2, 128, 217, 171), (0, 148, True)),
    ("list", 128, 16): ((4, 1, 12, 3, 128, 189, 178), (0, 148, True)),
    ("list", 128, 32): ((9, 1, 6, 2, 128, 166, 171), (0, 148, True)),
    # parts that follow the cache pass on all workers' multiprocessors
    ("turn", 64, 8): ((1, 1, 2, 2, 64, 684, 144), (6, 148, False)),
    ("turn", 64, 16): ((1, 5, 2, 1, 64, 772, 181), (7, 148, False)),
    ("turn", 64, 32): ((2, 4, 5, 1, 64, 159, 261), (2, 148, False)),
    ("turn", 64, 64): ((1, 5, 8, 1, 64, 185, 109), (2, 148, False)),
    ("turn", 128, 8): ((1, 1, 1, 1, 128, 585, 441), (5, 148, False)),
    ("turn", 128, 16): ((1, 2, 5, 1, 128, 590, 164), (5, 148, False)),
    ("turn", 128, 32): ((2, 4, 5, 1, 128, 185, 75), (2, 148, False)),
    ("turn", 128, 64): ((1, 5, 8, 1, 128, 201, 239), (2, 148, False)),
    # parts beside fewer workers
    ("beside", 64, 8): ((40, 1, 2, 2, 64, 142, 90), (2, 144, False)),
    ("beside", 64, 16): ((5, 4, 12, 4, 64, 134, 89), (2, 140, False)),
    ("beside", 64, 32): ((14, 5, 4, 1, 64, 130, 107), (2, 142, False)),
    ("beside", 64, 64): ((3, 5, 32, 4, 64, 142, 79), (2, 140, False)),
    ("beside", 128, 8): ((32, 1, 32, 8, 128, 8192, 1024), (5, 108, False)),
    ("beside", 128, 16): ((7, 5, 6, 3, 128, 136, 75), (2, 142, False)),
    ("beside", 128, 32): ((16, 5, 4, 1, 128, 147, 69), (2, 142, False)),
    ("beside", 128, 64): ((2, 5, 32, 4, 128, 157, 99), (2, 140, False)),
}


def lens_of(form):
    """Cache lengths of a form's case: empty, below the step's tokens, tile edges, full."""
    (B, steps, _, _, _, _, cap), _ = FORMS[form]
    rng = random.Random(repr(form))
    fixed = [cap, 65, 0, 64, 1]
    return [fixed[b] if b < len(fixed) else rng.randint(0, cap) for b in range(B)]
