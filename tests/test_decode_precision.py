"""The cases that show the bits of the attention's weights and queries are sharp (CPU): the documented
computation stays within their bounds, one with a term less does not."""

import numpy as np
import pytest

import oracle.decode as od
import precision_cases as pc


@pytest.mark.parametrize("f32_queries", [False, True])
@pytest.mark.parametrize("terms,holds", [(1, False), (2, False), (3, True)])
def test_the_weights_terms(f32_queries, terms, holds):
    q, k, v = pc.weight_case(1, 64, f32_queries)
    ref, _, _ = od.attn_ref(q[None], k[:, None], v[:, None], pc.TOKENS, 0.5)
    out, _ = pc.emulate(q, k, v, 0.5, 3, terms)
    err = np.abs(out - ref[0])
    assert (err <= pc.weight_bound(q, k, 0.5, ref[0])).all() == holds


@pytest.mark.parametrize("terms,holds", [(1, False), (2, False), (3, True)])
def test_the_queries_terms(terms, holds):
    q, k = pc.query_case(2, 64)
    _, ref, _ = od.attn_ref(q[None], k[:, None], k[:, None], 1, 0.7)
    _, lse = pc.emulate(q, k, k, np.float32(0.7), terms, 3)
    ref = ref[0] * (np.float64(np.float32(0.7)) / 0.7)
    assert (np.abs(lse - ref) <= pc.query_bound(ref)).all() == holds
