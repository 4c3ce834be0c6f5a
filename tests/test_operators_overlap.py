"""Refusal of an output that overlaps the queries (no GPU: fake device pointers, refused before any use)."""

import pytest

import paged_kv_cache_144_gb300 as pa

OTHER = 0x70000000
ROW = 8 * 128            # elements of a token's row


@pytest.fixture(scope="module")
def lib():
    return pa.load()


def _attend(lib, out, q, *, tokens=9, q_stride=ROW, out_dtype=pa.PA_BF16):
    """The status of a call that is right but for its pointers: PA_ERR_SHAPE when refused, else what the missing workspace
    or device gives."""
    return lib.pa_attend(out, out_dtype, q, pa.PA_BF16, q_stride, OTHER, 2 * OTHER, pa.PA_BF16, 100, None, None, OTHER, 16,
                         OTHER, OTHER, 4, tokens, 3, 8, 2, 128, 0.1, 16, None, 0, None, None)


Q = 0x10000000


@pytest.mark.parametrize("out,kw", [
    (Q, {}),                                                # the queries themselves
    (Q, dict(out_dtype=pa.PA_F32)),
    (Q, dict(tokens=1)),
    (Q + 9 * ROW * 2 - 16, {}),                             # the last chunk of the last row
    (Q - 9 * ROW * 2 + 16, {}),                             # out's last chunk
    (Q - 9 * ROW * 4 + 16, dict(out_dtype=pa.PA_F32)),
    (Q + ROW * 2, dict(q_stride=3 * ROW)),                  # out starts between rows and meets the next one
    (Q - 4 * ROW, dict(q_stride=100 * ROW)),                # around the first row
])
def test_an_output_over_the_queries_is_refused(lib, out, kw):
    assert _attend(lib, out, Q, **kw) == pa.PA_ERR_SHAPE


@pytest.mark.parametrize("out,kw", [
    (Q + 9 * ROW * 2, {}),                                  # right behind
    (Q - 9 * ROW * 2, {}),                                  # right before
    (Q - 9 * ROW * 4, dict(out_dtype=pa.PA_F32)),
    (Q + ROW * 2, dict(q_stride=10 * ROW)),                 # all of it in the gap behind the first row
    (Q + 2 * (4 * 10 * ROW + ROW), dict(q_stride=10 * ROW)),
    (Q + ROW * 2, dict(tokens=1, q_stride=2 * ROW)),
])
def test_an_output_beside_the_queries_is_not(lib, out, kw):
    assert _attend(lib, out, Q, **kw) != pa.PA_ERR_SHAPE
