"""What a long list asks for: the workspace of its largest table of 160 matrices,
as the tables follow one another; no GPU needed."""
import pytest


@pytest.fixture(scope="module")
def rr():
    from allgather_rr_allreduce_gb300 import build
    build.build()
    import allgather_rr_allreduce_gb300 as m
    return m


def of(rr, shapes):
    return rr.rr_orthogonalize_workspace([s[0] for s in shapes], [s[1] for s in shapes])


def test_tables_share_the_workspace(rr):
    a, b, none = (100, 300), (2000, 700), (0, 5)
    one_a, one_b = of(rr, [a]), of(rr, [b])
    assert of(rr, [a] * 160) == 160 * one_a
    assert of(rr, [a] * 161) == of(rr, [a] * 480) == 160 * one_a
    assert of(rr, [a] * 160 + [b] * 40) == max(160 * one_a, 40 * one_b)
    assert of(rr, [b] * 40 + [a] * 160) == 40 * one_b + 120 * one_a
    # empty matrices take no place in a table
    assert of(rr, [none] * 50 + [a] * 100 + [none] * 50 + [a] * 60 + [b]) == max(160 * one_a, one_b)
