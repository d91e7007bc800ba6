"""Searches whose rows are more than a step's streams or a reordering's caches: each selection takes them all, its parents
number rows of the whole call, and tfl_kv_reorder_rows moves a group's caches by them."""
import pytest
import torch

from gqa_decoder_forward_gb300 import build, synth, tfl
from tests import beam_ref
from tests.test_gpu_beam_select import plain_model
from tests.test_gpu_kv_reorder import filled, pages
from tests.test_gpu_shared_model import GATE, MAXP, S, ids_of, logits_of, prompt, tails_of

pytestmark = pytest.mark.gpu
INT = torch.iinfo(torch.int32)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    build.build()


@pytest.mark.parametrize("first,parents", [
    (16, [17, 16]), (48, [50, 48, 49, 48, 63]), (5, [4, 5, 0, 10, -1, INT.min, INT.max, 6]), (INT.max - 2, [INT.max, INT.max - 2, INT.min]),
    (16, list(range(31, 15, -1))), (16, list(range(16)))])
def test_moves_by_the_rows_of_a_larger_call(first, parents):
    m = plain_model(S, 16, 300)
    n = len(parents)
    kvs = filled(m, n, 300, 610)
    old = [pages(m, kv, 300).clone() for kv in kvs]
    tfl.tfl_kv_reorder_rows(m, tfl.KVRows(kvs, [120] * n, [11] * n), first, torch.tensor(parents, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for i, p in enumerate(parents):
        want = old[i].clone()
        if first <= p < first + n:
            want[:, :, 120: 131] = old[p - first][:, :, 120: 131]
        assert torch.equal(pages(m, kvs[i], 300), want), i


def test_refusals():
    m = plain_model(S, 16, 300)
    batch = tfl.KVRows(filled(m, 2, 300, 611), [0, 0], [1, 1])
    parents = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    with pytest.raises(tfl.TflError) as e:
        tfl.tfl_kv_reorder_rows(m, batch, -1, parents)
    assert e.value.code == tfl.TFL_E_ARG
    with pytest.raises(ValueError):
        tfl.tfl_kv_reorder_rows(m, batch, 2 ** 32, parents)


@pytest.mark.parametrize("length,groups", [(200, 2), (77, 4)])
def test_searches_of_sixteen_beams(length, groups):
    """As a program runs them: a step per search, one selection, a reordering per search; each selection against 64 bits, and
    the kept beams' last logits against a fresh prompt of their tokens."""
    m = tfl.Model(S, synth.model_weights(S, 61, "cuda"), max_rows=512, max_decode_rows=64, max_context=MAXP)
    runner, beams, steps = tfl.SharedRunner(m), 16, 5
    n = groups * beams
    prefixes, firsts = zip(*[prompt(m, length, 620 + g) for g in range(groups)])
    tails = [tails_of(m, kv, beams) for kv in prefixes]
    batches = [tfl.SharedRows([kv], [beams], t) for kv, t in zip(prefixes, tails)]
    ranges = [tfl.KVRows(t, [length % 128] * beams, [0] * beams) for t in tails]
    new = lambda t: torch.zeros(groups, beams, dtype=t, device="cuda")  # noqa: E731
    ids, parents, scores, logits = new(torch.int32), new(torch.int32), new(torch.float32), logits_of(n)
    seen = []

    def select(z, s):
        before = z.clone(), s.clone()
        tfl.tfl_beam_select(m, z, s, ids, parents, scores)
        seen.append((*before, ids.clone(), parents.clone()))

    select(torch.cat(firsts), torch.zeros(groups, 1, device="cuda"))
    for step in range(steps):
        for g in range(groups):
            runner.decode_step(batches[g], ids[g], logits[g * beams: (g + 1) * beams])
        select(logits, scores)
        for g in range(groups):
            ranges[g].set([length % 128] * beams, [step + 1] * beams)
            tfl.tfl_kv_reorder_rows(m, ranges[g], g * beams, parents[g])
    torch.cuda.synchronize()
    assert m.status() == tfl.TFL_OK

    said = []
    for k, (z, s, got_ids, got_parents) in enumerate(seen):
        want = beam_ref.select(z.double().cpu().numpy(), s.double().cpu().numpy(), beams)
        assert (got_ids.cpu().numpy() == want[0]).all() and (got_parents.cpu().numpy() == want[1]).all()
        said = [(said[p] if k else []) + [v] for p, v in zip(got_parents.view(-1).tolist(), got_ids.view(-1).tolist())]
    z, last = seen[-1][0], seen[-1][3].view(-1).tolist()
    assert any(p % beams != i % beams for i, p in enumerate(last))   # caches have moved
    for i in range(n):
        fresh, out = m.kv(MAXP), logits_of(1)
        text = torch.cat((ids_of(620 + i // beams, length), torch.tensor(said[i][:-1], dtype=torch.int32, device="cuda")))
        m.prefill_chunk(fresh, text, out)
        assert (out[0].float() - z[last[i]].float()).abs().max() <= GATE, i
