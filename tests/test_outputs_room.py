"""Outputs that a caller gives must have room for what is written: refused before any
call, so no GPU is needed (the tensors are the host's, the library a stand-in)."""
import pytest
import torch

from model_free_suffix_gb300 import Proposal, SuffixDrafter, Verdict

B, K, V = 4, 3, 50


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def dr():
    d = SuffixDrafter.__new__(SuffixDrafter)
    d._lib, d._h = Library(), None
    d._index, d.device = -1, torch.device("cpu")
    d.k, d.V, d.S, d.max_batch = K, V, 64, 8
    return d


def _verify(dr, out):
    i32 = dict(dtype=torch.int32)
    return dr.verify(torch.zeros(B * (K + 1), V), torch.zeros(B, K, **i32), torch.zeros(B, **i32), torch.zeros(B, K),
                     torch.ones(B, V), out=out, stream=0)


def test_verdict_of_too_small_a_batch_or_another_width(dr):
    full = dr.new_verdict(B)
    small, wide, narrow = dr.new_verdict(B - 1), dr.new_verdict(B + 2), dr.new_verdict(B)
    narrow.sampled, narrow.logprobs = narrow.sampled[:, :K].contiguous(), narrow.logprobs[:, :K].contiguous()
    bad = [small, narrow] + [Verdict(*(o if i == j else f for j, (o, f) in enumerate(zip(vars(w).values(), vars(full).values()))))
                             for w in (small, narrow) for i in range(3) if w is small or i != 1]
    bad += [Verdict(full.sampled.view(-1), full.num_accepted, full.logprobs),
            Verdict(full.sampled, full.num_accepted[:, None], full.logprobs)]
    for v in bad:
        with pytest.raises(ValueError):
            _verify(dr, v)
    assert dr._lib.calls == []
    for v in (full, wide, Verdict(full.sampled, full.num_accepted, None)):
        assert _verify(dr, v) is v
    assert dr._lib.calls == ["sgd_verify"] * 3


I32 = dict(dtype=torch.int32)


def _drafting_calls(dr, out):
    tok, n, sampled, doc = torch.zeros(B, 64, **I32), torch.zeros(B, **I32), torch.zeros(B, 2, **I32), torch.zeros(1, **I32)
    h = (out.drafts, out.num_valid, out.score, out.probs, out.match_info)
    return [lambda: dr.propose(tok, n, out=out, stream=0),
            lambda: dr.propose_with_update(tok, n, sampled, out=out, stream=0),
            lambda: dr.step(tok, n, sampled, doc, doc, doc, out=out, stream=0),
            lambda: dr.step_host(tok, n, sampled, doc, doc, doc, *h, stream=0),
            lambda: dr.bind_step_host(tok, n, sampled, doc, doc, doc, *h, stream=0)]


def test_proposal_of_too_small_a_batch_or_width(dr):
    full, small = vars(dr.new_outputs(B)), vars(dr.new_outputs(B - 1))
    dr.k = K - 1
    narrow = vars(dr.new_outputs(B))
    dr.k = K
    for name in full:
        for other in (small, narrow):
            if other[name].numel() < full[name].numel():
                for f in _drafting_calls(dr, Proposal(**dict(full, **{name: other[name]}))):
                    with pytest.raises(ValueError):
                        f()
    assert dr._lib.calls == []
    for out in (Proposal(**full), dr.new_outputs(B + 3),
                Proposal(full["drafts"], full["num_valid"], None, None, None),
                Proposal(**{name: t.view(-1) for name, t in full.items()})):
        for f in _drafting_calls(dr, out):
            f()
    assert len(dr._lib.calls) == 4 * 4   # (a bound step is not called yet)
