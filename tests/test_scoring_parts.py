"""How few long rows are cut, on the CPU, from the workspaces that the library asks for: no part lies past its row."""
import ctypes as C
import random

import pytest

pytest.importorskip("torch")

from byte_level_bpe_amd import scoring  # noqa: E402

PARTIAL, SCORE = 16, 24  # bytes of a part's numbers


def parts_of(dtype, rows, vocab, k):
    """Parts of a row as distillation's loss and as scores cut it, 1 where it is whole."""
    n, lib = C.c_uint64(), scoring._lib()
    assert lib.bbpe_distill_loss_workspace_bytes(dtype, rows, vocab, C.byref(n)) == 0 and n.value % (rows * PARTIAL) == 0
    found = [n.value // (rows * PARTIAL)]
    assert lib.bbpe_token_logprobs_workspace_bytes(dtype, rows, vocab, k, C.byref(n)) == 0
    p = n.value // (rows * (SCORE + 8 * k))
    if k:  # the numbers are rounded up to 256 bytes
        p = next((q for q in range(64, 0, -1) if (rows * q * SCORE + 255) // 256 * 256 + rows * q * k * 8 == n.value), 0)
    found.append(p)
    return [max(1, p) for p in found]


def test_no_part_past_the_row():
    rng = random.Random(7)
    cases = [(2, 17, 249854, 0), (2, 128, 200005, 20), (0, 8, 100277, 5)]
    for _ in range(3000):
        cases.append((rng.choice([0, 1, 2]), rng.randint(1, 600), int(2 ** rng.uniform(11, 20)), rng.choice([0, 0, 1, 20, 200])))
    cut = 0
    for dtype, rows, vocab, k in cases:
        each = 4 if dtype == 2 else 8
        pieces = (vocab + 2 * (each - 1)) // each  # wherever it begins
        for parts in parts_of(dtype, rows, vocab, k):
            part = (-(-pieces // parts) + 63) // 64 * 64
            assert (parts - 1) * part < pieces, (dtype, rows, vocab, k, parts, part)
            cut += parts > 1
    assert cut > 1000
