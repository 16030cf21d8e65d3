"""The nodes of a drafted step from a draft's tokens (host bookkeeping)."""
import pytest

from invariant_forward_policy_gb300.decoder import draft_nodes


def test_the_last_token_is_node_zero():
    assert draft_nodes([], [], 7, 5, 8) == ([7], [-1])
    assert draft_nodes([1, 2, 3], [-1, 0, -1], 7, 5, 8) == ([7, 1, 2, 3], [-1, 0, 1, 0])


def test_deep_and_surplus_drafts_go_with_what_hangs_on_them():
    # room for 2 tokens: the last token's choice and one draft's
    assert draft_nodes([1, 2, 3, 4], [-1, 0, -1, 1], 7, 2, 8) == ([7, 1, 3], [-1, 0, 0])
    assert draft_nodes([1, 2], [-1, 0], 7, 1, 8) == ([7], [-1])
    assert draft_nodes([1, 2, 3], [-1, -1, 1], 7, 9, 2) == ([7, 1], [-1, 0])


def test_refusals():
    for toks, pars in (([1], [0]), ([1], [-2]), ([1, 2], [-1, 1]), ([1], [])):
        with pytest.raises(ValueError):
            draft_nodes(toks, pars, 7, 5, 8)
