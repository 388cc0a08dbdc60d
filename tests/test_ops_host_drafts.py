"""What the entry points for drafts and bounded caches refuse before they touch a device (no GPU needed)."""
import pytest

from latency_moe_decode_gb300 import capi
from latency_moe_decode_gb300.capi import (DecDraftTreeArgs, DecKvqHeaviestArgs, DecKvqMassArgs, DecKvqMoveArgs,
                                           DecVerifyDraftsArgs)
from test_ops_host import ARG, UNSUPPORTED, _attn, _cache, _flat, _r, _seqs, lib  # noqa: F401


def _tree(**kw):
    d = dict(batch=1, n_tokens=8, cu_tokens=4096, parents=4096, lengths=4096, max_tokens=8, mask=4096, mask_stride=1,
             positions=4096)
    d.update(kw)
    return DecDraftTreeArgs(**d)


def _mass(**kw):
    d = dict(n_heads=8, q=_r(), lse=4096, causal=1, max_tokens=1, decay=1.0, mass=4096, mass_out=4096)
    d.update(kw)
    return DecKvqMassArgs(**_flat(d))


def _keep(**kw):
    d = dict(mass=4096, budget=64, sinks=4, recent=16, kept=4096, count=4096)
    d.update(kw)
    return DecKvqHeaviestArgs(**d)


def _move(**kw):
    d = dict(index=4096, index_stride=64, head_stride=0, count=4096, max_count=64)
    d.update(kw)
    return DecKvqMoveArgs(**d)


def _verify(**kw):
    d = dict(logits=4096, dtype=1, vocab=1000, row_stride=1000, draft_probs=4096, prob_stride=1000, batch=2, n_tokens=8,
             cu_tokens=4096, tokens=4096, parents=4096, uniforms=4096, temperature=4096, max_tokens=4, path=4096, count=4096,
             next_tokens=4096, workspace=4096, workspace_bytes=1 << 20)
    d.update(kw)
    return DecVerifyDraftsArgs(**d)


@pytest.mark.parametrize("args,status", [
    (None, ARG), (dict(batch=-1), ARG), (dict(n_tokens=-1), ARG), (dict(max_tokens=-1), ARG), (dict(max_tokens=1025), UNSUPPORTED),
    (dict(cu_tokens=None), ARG), (dict(parents=None), ARG), (dict(mask=None), ARG), (dict(lengths=None), ARG),
    (dict(max_tokens=33), ARG), (dict(mask_stride=-1), ARG), (dict(mask=4098), ARG)])
def test_draft_trees_are_checked(lib, args, status):  # noqa: F811
    assert lib.dec_draft_tree(None if args is None else _tree(**args), None) == status
    assert b"draft_tree" in lib.dec_op_error()
    assert lib.dec_draft_tree(_tree(batch=0, n_tokens=0, parents=None, mask=None, cu_tokens=None), None) == 0


@pytest.mark.parametrize("args,status", [
    (dict(causal=0, tree_mask=4096, tree_words=1, tree_stride=1), ARG), (dict(tree_mask=4096, tree_words=0), ARG),
    (dict(tree_mask=4096, tree_words=33, tree_stride=33), UNSUPPORTED), (dict(tree_mask=4096, tree_words=1, tree_stride=-1), ARG),
    (dict(tree_mask=4098, tree_words=1, tree_stride=1), ARG)])
def test_tree_masks_are_checked(lib, args, status):  # noqa: F811
    assert lib.dec_kvq_attention(_cache(), _seqs(), _attn(workspace=4096, workspace_bytes=1 << 40, **args), None) == status
    assert b"tree" in lib.dec_op_error()


@pytest.mark.parametrize("args,status", [
    (None, ARG), (dict(n_heads=0), ARG), (dict(n_heads=7), ARG), (dict(max_tokens=-1), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG), (dict(decay=float("nan")), ARG), (dict(decay=float("inf")), ARG),
    (dict(q=_r(p=None)), ARG), (dict(q=_r(head_stride=4)), ARG), (dict(lse=None), ARG), (dict(mass=None), ARG),
    (dict(mass_out=None), ARG), (dict(mass=4098), ARG), (dict(lse=4097), ARG)])
def test_masses_are_checked(lib, args, status):  # noqa: F811
    assert lib.dec_kvq_mass(_cache(), _seqs(), None if args is None else _mass(**args), None) == status
    assert b"mass" in lib.dec_op_error()
    assert lib.dec_kvq_mass(_cache(), _seqs(batch=0, n_tokens=0), _mass(), None) == 0


@pytest.mark.parametrize("args,status", [
    (None, ARG), (dict(budget=0), ARG), (dict(sinks=-1), ARG), (dict(recent=-1), ARG), (dict(sinks=40, recent=25), ARG),
    (dict(mass=None), ARG), (dict(kept=None), ARG), (dict(count=None), ARG), (dict(kept=4098), ARG),
    (dict(budget=2 ** 31 - 5), UNSUPPORTED)])
def test_choices_are_checked(lib, args, status):  # noqa: F811
    assert lib.dec_kvq_heaviest(_cache(), _seqs(), None if args is None else _keep(**args), None) == status
    assert b"heaviest" in lib.dec_op_error()


@pytest.mark.parametrize("args,status", [
    (None, ARG), (dict(max_count=-1), ARG), (dict(index_stride=-1), ARG), (dict(head_stride=-1), ARG), (dict(index=None), ARG),
    (dict(count=None), ARG), (dict(index=4098), ARG), (dict(mass=4098), ARG), (dict(to=4096, to_pages=0), ARG),
    (dict(to=4096, to_pages=1, to_stride=-1), ARG), (dict(to=4096, to_pages=1 << 26), UNSUPPORTED),
    (dict(max_count=2 ** 31 - 1), UNSUPPORTED)])
def test_moves_are_checked(lib, args, status):  # noqa: F811
    assert lib.dec_kvq_move(_cache(), _seqs(), None if args is None else _move(**args), None) == status
    assert b"move" in lib.dec_op_error()
    assert lib.dec_kvq_move(_cache(), _seqs(), _move(max_count=0), None) == 0


def test_sequences_with_token_rows_are_refused(lib):  # noqa: F811
    rows = dict(cu_tokens=4096, n_tokens=3)
    assert lib.dec_kvq_heaviest(_cache(), _seqs(**rows), _keep(), None) == ARG
    assert lib.dec_kvq_move(_cache(), _seqs(**rows), _move(), None) == ARG
    assert lib.dec_kvq_heaviest(_cache(), _seqs(lengths=None), _keep(), None) == ARG
    for bad in (dict(pages=None), dict(head_dim=96), dict(page_tokens=24)):
        assert lib.dec_kvq_heaviest(_cache(**bad), _seqs(), _keep(), None) != 0
        assert lib.dec_kvq_move(_cache(**bad), _seqs(), _move(), None) != 0
        assert lib.dec_kvq_mass(_cache(**bad), _seqs(), _mass(), None) != 0


@pytest.mark.parametrize("args,status", [
    (None, ARG), (dict(dtype=2), ARG), (dict(vocab=0), ARG), (dict(batch=-1), ARG), (dict(n_tokens=-1), ARG), (dict(max_tokens=-1), ARG),
    (dict(row_stride=-1), ARG), (dict(prob_stride=-1), ARG), (dict(max_tokens=1025), UNSUPPORTED), (dict(logits=None), ARG),
    (dict(tokens=None), ARG), (dict(uniforms=None), ARG), (dict(cu_tokens=None), ARG), (dict(path=None), ARG), (dict(count=None), ARG),
    (dict(next_tokens=None), ARG), (dict(workspace=None), ARG), (dict(workspace=4100), ARG), (dict(workspace_bytes=100), ARG),
    (dict(logits=4098), ARG), (dict(draft_probs=4098), ARG), (dict(vocab=2 ** 24 + 1), UNSUPPORTED), (dict(n_tokens=2 ** 30), UNSUPPORTED)])
def test_verifications_are_checked(lib, args, status):  # noqa: F811
    assert lib.dec_verify_drafts(None if args is None else _verify(**args), None) == status
    assert b"verify_drafts" in lib.dec_op_error()
    assert lib.dec_verify_drafts(_verify(batch=0), None) == 0
    assert lib.dec_verify_drafts_workspace(8) > 0 and lib.dec_verify_drafts_workspace(-1) == -1


def test_tensors_are_checked():
    """The torch binding's own refusals that need no device."""
    import torch

    from latency_moe_decode_gb300 import ops
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.draft_tree(i32(4), i32(1), i32(2))
    with pytest.raises(ValueError):
        ops.verify_drafts(torch.zeros(4, 8), i32(4), torch.zeros(4), i32(2))
    assert capi.DEC_MAX_TREE == 1024
