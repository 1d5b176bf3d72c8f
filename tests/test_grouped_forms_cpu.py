"""The sizes of the GPU tests of every form (experts_cases.FORMS) reach, on a card of
256 compute units, every kernel of the grouped products in every form that it has:
tile, gated or not, rows gathered or not.  Counted are the calls that those tests
make, not sizes alone."""
import itertools

import experts_cases as C
from test_grouped_plan_cpu import DW, DX, FWD, SKINNY, STREAM, TILE_128, TILE_128x256, TILE_256, plan  # noqa: F401

BOTH = (False, True)


def _calls():
    for (counts, behind, K, O), act, gather in itertools.product(C.FORMS, C.FORM_ACTS, BOTH):
        glu = act == "swiglu"
        yield sum(counts) + behind, len(counts), 2 * O if glu else O, K, glu, gather


def test_every_form_of_the_bf16_products(plan):  # noqa: F811
    seen = {(plan.bf16(FWD, *s), glu, gather) for *s, glu, gather in _calls()}
    assert seen == set(itertools.product((TILE_256, TILE_128, SKINNY), BOTH, BOTH))
    assert {plan.bf16(DX, *s) for *s, _, _ in _calls()} == {TILE_256, TILE_128, TILE_128x256, STREAM}
    # a weight gradient's rows are gathered by the launch before it
    seen = {(t, t == TILE_128 and plan.splits(*s) > 1, gather) for *s, _, gather in _calls() for t in [plan.bf16(DW, *s)]}
    assert seen == set(itertools.product((TILE_256, STREAM), (False,), BOTH)) | set(itertools.product((TILE_128,), BOTH, BOTH))


def test_every_form_of_the_fp32_products(plan):  # noqa: F811
    seen = {(plan.f32(FWD, *s), glu, gather) for *s, glu, gather in _calls()}
    assert seen == set(itertools.product((32, 64, 128), BOTH, BOTH))
    assert {plan.f32(DX, *s) for *s, _, _ in _calls()} == {32, 64, 128}
    assert {(plan.f32(DW, *s), gather) for *s, _, gather in _calls()} == set(itertools.product((32, 64, 128), BOTH))
    pair = {gather for *s, _, gather in _calls() if plan.f32(DX, *s) == plan.f32(DW, *s) == 32}  # one launch for both
    assert pair == set(BOTH)


def test_few_rows_reach_the_panels_edges(plan):  # noqa: F811
    """Experts of no, one, up to 16 and more rows, reductions that 64 does not divide
    and, of 16 weight rows, a last panel that is cut."""
    few = [(counts, K, O) for (counts, behind, K, O), act in itertools.product(C.FORMS, C.FORM_ACTS)
           if plan.bf16(FWD, sum(counts) + behind, len(counts), 2 * O if act == "swiglu" else O, K) == SKINNY]
    rows = {n for counts, _, _ in few for n in counts}
    assert 0 in rows and 1 in rows and any(1 < n < 16 for n in rows) and any(n > 32 for n in rows)
    assert any(K % 64 for _, K, _ in few) and any(O % 16 for _, _, O in few)
