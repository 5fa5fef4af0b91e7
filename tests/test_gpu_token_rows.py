"""The mixers' token steps where a CTA has several rows, as a full batch has:
delta rule with two rows a CTA ([dk, dv] states) and two to four ([dv, dk]
ones), the conv with two to four groups of rows, against the fp64 oracle: rows
of one slot inside a CTA, next to one another and in turn, in several CTAs,
empty rows among them, in place and into another pool.
"""
import pytest
import torch

from test_gpu_token_step import _cuda, check_conv, check_delta, conv_case, draw_delta, run_delta  # noqa: F401  (_cuda: the GPU or a skip)

pytestmark = pytest.mark.gpu


def rows_of_a_cta(n, slices, per_sm, most):
    """As launch_g chooses: several rows for a CTA as long as two waves of CTAs are left."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return max(1, min(most, n * slices // (2 * sms * per_sm)))


def batch(slices, per_sm, rows):
    """The smallest odd batch whose CTAs have `rows` rows each."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = -(-rows * 2 * sms * per_sm // slices)
    return n + 1 - n % 2


def slots_of(order, n):
    gen = torch.Generator().manual_seed(n)
    if order == "one each":
        return torch.randperm(n + 3, generator=gen)[:n].tolist()
    if order == "next to one another":          # i // 3: runs begin at every place of a CTA
        return [i // 3 for i in range(n)]
    if order == "in turn inside a CTA":         # a b a b
        return [i // 4 * 2 + i % 2 for i in range(n)]
    if order == "in turn":                      # every CTA but the first ones has only rows that others take along
        return [i % 29 for i in range(n)]
    t = torch.randint(-1, n // 3, (n,), generator=gen)     # in no order, with empty rows
    t[::11] = n // 3 + 5                                     # and slots past the pool
    return t.tolist()


ORDERS = ["one each", "next to one another", "in turn inside a CTA", "in turn", "in no order"]


@pytest.mark.parametrize("order", ORDERS)
def test_two_rows_of_kfirst_states(order):
    H, d = 8, 64
    n = batch(H, 4, 2)
    assert rows_of_a_cta(n, H, 4, 2) == 2
    slots = slots_of(order, n)
    S = n // 3 if order == "in no order" else max(slots) + 2
    for dtype, gate, G, in_place in (("bf16", "gdn", 1, True), ("fp32", "kda", 2, False)):
        case = draw_delta(n, H, G, d, gate, dtype, S, seed=len(order))
        o, out = run_delta(case, slots, dtype, gate, False, in_place=in_place, G=G)
        check_delta(case, slots, o, out, dtype, fill=None if in_place else 99.0)


@pytest.mark.parametrize("rows", [2, 3, 4])
@pytest.mark.parametrize("order", ORDERS)
def test_several_rows_of_vfirst_states(order, rows):
    H, d = 8, 64
    for dtype, gate, G, per_sm, in_place in (("bf16", "gdn", 1, 5, True), ("fp32", "kda", 2, 4, False)):
        n = batch(H * 2, per_sm, rows)
        assert rows_of_a_cta(n, H * 2, per_sm, 4) == rows
        slots = slots_of(order, n)
        S = n // 3 if order == "in no order" else max(slots) + 2
        case = draw_delta(n, H, G, d, gate, dtype, S, seed=rows)
        o, out = run_delta(case, slots, dtype, gate, True, in_place=in_place, G=G)
        check_delta(case, slots, o, out, dtype, fill=None if in_place else 99.0)


@pytest.mark.parametrize("vfirst", [False, True])
def test_a_full_batch_of_wide_heads(vfirst):
    """d = 128 and 16 heads: the token that follows one another's slot in the same CTA, and rows without slots."""
    H, d = 16, 128
    n = batch(H * (4 if vfirst else 2), 5 if vfirst else 3, 4 if vfirst else 2)
    S = n + 1
    case = draw_delta(n, H, 1, d, "gdn", "bf16", S, seed=3)
    slots = [-1 if i % 17 == 5 else i // 2 for i in range(n)]
    o, out = run_delta(case, slots, "bf16", "gdn", vfirst)
    check_delta(case, slots, o, out, "bf16")
    o, out = run_delta(case, None, "bf16", "gdn", vfirst)
    check_delta(case, None, o, out, "bf16")


@pytest.mark.parametrize("vfirst", [False, True])
def test_long_batches_of_tokens_in_turn(vfirst):
    """More rows than one look of the search: 1500 tokens of 5 sequences in turn, one sequence's first token last."""
    n = 1501
    slots = [i % 5 for i in range(n - 1)] + [6]
    slots[700:1300] = [-1] * 600
    case = draw_delta(n, 1, 1, 64, "kda", "fp32", 8, seed=1)
    o, out = run_delta(case, slots, "fp32", "kda", vfirst)
    check_delta(case, slots, o, out, "fp32")


# ------------------------------------------------------------------ conv
def conv_batch(dtype, channels, groups):
    """The smallest odd batch whose CTAs have `groups` groups of rows each (conv_w's choice)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows, blocks = 4 if dtype == "bf16" else 2, -(-channels // 512)
    return rows * -(-groups * 8 * sms // blocks) - 1


@pytest.mark.parametrize("groups", [2, 3, 4])
@pytest.mark.parametrize("order", ORDERS)
def test_several_groups_of_conv_rows(order, groups):
    for dtype, W, act, bias, in_place in (("bf16", 4, "silu", True, True), ("fp32", 3, None, False, False)):
        C = 6152                                   # the last CTA of a row has two threads with channels
        n = conv_batch(dtype, C, groups)
        slots = slots_of(order, n)
        S = n // 3 if order == "in no order" else max(slots) + 2
        check_conv(conv_case(n, C, W, S, dtype, seed=groups), slots, dtype, act, bias, in_place)


def test_conv_groups_without_slots():
    n = conv_batch("bf16", 6152, 4)
    check_conv(conv_case(n, 6152, 4, n + 1, "bf16"), None, "bf16")


def test_conv_long_batches_of_tokens_in_turn():
    n = 1501
    slots = [i % 5 for i in range(n - 1)] + [6]
    slots[700:1300] = [-1] * 600
    check_conv(conv_case(n, 40, 4, 8, "bf16"), slots, "bf16")
