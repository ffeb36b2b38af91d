"""The calls of a verify step together (examples/verify_step.py): tokens fed
as a drafted tree give the logits that their branches give when decoded token
by token, over either cache type."""
import os
import sys

import pytest
import torch

from tests.gpu_util import need_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (16, 1, 128)])
def test_a_tree_scores_its_branches_as_decoding_does(cache, Hq, Hkv, D):
    import verify_step as vs
    model = vs.Model(Hq=Hq, Hkv=Hkv, D=D, cache=cache, seed=3)
    i32 = dict(dtype=torch.int32, device="cuda")
    prompt = [29, 50]
    tokens = torch.randint(0, model.vocab, (79,), generator=torch.Generator().manual_seed(1)).cuda()
    drafted = torch.randint(0, model.vocab, (5,), generator=torch.Generator().manual_seed(2)).cuda()
    parents, depth = [-1, 0, 1, 0, 3], [0, 1, 2, 1, 2]
    bits = [1, 3, 7, 9, 25]

    def prefill():
        free, table = torch.arange(256, **i32), torch.full((2, 16), -1, **i32)
        context, new = torch.zeros(2, **i32), torch.tensor(prompt, **i32)
        places = vs.place(context, new, free, table, model.page)
        model.step(tokens, places, table, context, None)
        return free[int(places["counts"][1]):], table, context + new

    free, table, context = prefill()
    new = torch.tensor([5, 5], **i32)
    places = vs.place(context, new, free, table, model.page, torch.tensor(depth * 2, **i32))
    mask = torch.tensor(bits * 2, device="cuda")[:, None].contiguous()
    tree = model.step(drafted.repeat(2), places, table, context, mask)

    for leaf in (2, 4):
        path = [leaf]
        while parents[path[0]] >= 0:
            path.insert(0, parents[path[0]])
        free, table, context = prefill()
        for j in path:
            new = torch.ones(2, **i32)
            places = vs.place(context, new, free, table, model.page)
            one = model.step(drafted[[j, j]], places, table, context, None)
            free, context = free[int(places["counts"][1]):], context + new
            for r in range(2):
                want, got = one[r], tree[5 * r + j]
                # both are sums over the same bf16 (or E4M3) cache; attention's bf16 roundings (2^-8 of values of
                # about 1) pass two projections of unit gain
                assert (got - want).abs().max() < 0.1 and (got - want).norm() / want.norm() < 0.01, (leaf, j, r)
    lp, entropy, ids, top = vs.score(tree, drafted.repeat(2).to(torch.int32))
    ref = torch.log_softmax(tree.double(), 1)
    assert torch.allclose(lp.double(), ref[torch.arange(10), drafted.repeat(2)], atol=1e-3)
    assert torch.equal(ids.long(), ref.topk(4, 1).indices)


def test_the_example_runs(capsys):
    import verify_step as vs
    vs.main()
    assert capsys.readouterr().out.count("log probability") == 8
